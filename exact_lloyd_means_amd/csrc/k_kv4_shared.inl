// k_kv4_shared.inl -- attention of requests that share a prefix
// (fk_kv4_attention_shared), on the waves of k_kv4_attn.inl.
//
// The query rows of a group's requests lie one after another, so 16 NA of them
// make a tile that walks the prefix once, whatever requests they belong to: for
// single tokens a tile serves 16 NA / G requests instead of one, and a block's
// codes are read and looked up that many times less.  What lies behind the
// prefix is walked for each request as in the split form.  Two launches:
//
//   k_kv4_shared_walk  segments of the tiles' keys (one a workgroup) and shares of
//                      the requests' own keys (one a wave), as many workgroups for
//                      each as let them end together; those whose segment is over
//                      earlier take shares too; sums of rows go to the workspace
//   k_kv4_shared_join  adds up the segments and shares of each request, in order
//
// 64 requests of 16-600 tokens behind 8192 shared ones, 32 / 8 heads of 128: 36.8 us
// a call (as plain attention 82; the two launches take 40 when traced).  Of a
// workgroup's 30 us in the walk 6 pass until it knows its work, 3.5 until its codes
// are there, 14 to 20 with the 10 or 11 blocks of a wave, 3 with adding up its
// waves; the join takes 5.  Eight groups of sixteen behind 1000-6000, 64 / 8 heads,
// 122 MB of codes: 66 us (85).  Memory alone would take 26 of them and the vector
// instructions 24 (13 of the 36.8): two waves a SIMD, as many as the registers
// leave, hide neither behind the other.
//
// Tried: the plan as a launch of its own (44 us against 41, before later steps),
// pieces of the line of all tiles instead of segments of each (a workgroup in two
// tiles pays both ends: 8 x 16 63 -> 75), more workgroups than run at once (37 ->
// 50), 32 rows a wave of 256 dimensions at one wave a SIMD (82 -> 98 for 180
// requests).
#pragma once

#include "k_kv4_attn.inl"
#include "serve_internal.h"

namespace fk {
namespace {

// What balances the two kinds of work, in tenths of a microsecond at two waves a
// SIMD with heads of 128: a block of 16 NT rows; what a segment costs beside its
// blocks (codes on their way, waves added up); a unit of a share likewise, in
// blocks of its own.
template <int NT>
constexpr int kBlockTime = 3 + 5 * NT;
template <int NT>
constexpr int kOwnTime = NT < 2 ? 13 : kBlockTime<NT>;
constexpr int kSegmentTime = 140, kShareTime = 80, kAgainTime = 60;  // a share behind a segment
constexpr int kUnitBlocks = kSharedUnit;

// Row tiles of requests.
__device__ inline Span own_span(const AttnArgs& a, Rows& rw, int rt, int rows, int prefix) {
    Span sp = tile_rows(a, rw, rt * rows, rows);
    sp.lo = sp.lo > prefix ? sp.lo : prefix;
    sp.hi = sp.hi > sp.lo ? sp.hi : sp.lo;
    return sp;
}

// build_table in two steps: the codebook's row of the thread's column is on its
// way while lengths are.
struct Codebook {
    uintx4 x[2];
    __device__ inline void load(const AttnArgs& a, int h, int tid) {
        const uintx4* p = reinterpret_cast<const uintx4*>(a.codebook + ((tid >> 3 & 1) * a.Hkv + h) * 16);
        x[0] = p[0];
        x[1] = p[1];
    }
    __device__ inline void build(uint32_t* tab, int tid) const {
        const int col = tid & 15, lo = tid >> 4 & 15;
        uint32_t low = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t v = x[i >> 3][i >> 1 & 3] >> (16 * (i & 1)) & 0xffffu;
            low = lo == i ? v : low;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t v = low | (x[i >> 3][i >> 1 & 3] >> (16 * (i & 1)) & 0xffffu) << 16;
            *reinterpret_cast<uintx4*>(tab + (i * 16 + lo) * 64 + col * 4) = uintx4{v, v, v, v};
        }
    }
};

struct SharedGroup {  // in LDS
    int req0, req1;   // its requests
    int tok0, rows;   // their first query token and their query rows
    int blocks;       // of the prefix, 0: nothing is shared
    int lo, len;      // blocks that some row sees (first: first and last position)
    int base;         // its first segment
    int mixed;        // some row does not see all of the prefix's blocks
    int pad[3];
};

// The group of request b, -1: none.
__device__ inline int group_of(const SharedGroup* g, int groups, int b) {
    int lo = 0, hi = groups;  // g[lo].req0 <= b < g[hi].req0
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (g[mid].req0 <= b) lo = mid;
        else hi = mid;
    }
    // of empty groups at one place the last is found: it is the one that may hold b
    return b >= g[lo].req0 && b < g[lo].req1 && g[lo].blocks > 0 ? lo : -1;
}

// What a wave starts with: a unit, and its place in the line.
struct Start {
    int unit, at;
};

struct Shares {
    int segments;  // of all groups; workgroups from the first on take one each
    int seg_len;   // most blocks of one
    int total;     // the line of units: kUnitBlocks and the own blocks of each
    // What a wave takes of it, the last workgroup's waves first: `share` each of
    // `border` waves, `extra` each of those that had a segment before.
    int share, extra, border;
    __device__ inline int64_t begin(int w) const {
        return w <= border ? (int64_t)w * share : (int64_t)border * share + (int64_t)(w - border) * extra;
    }
    __device__ inline int wave_of(int64_t at) const {
        const int64_t rest = at - (int64_t)border * share;
        return rest < 0 ? (int)at / share : border + (int)rest / extra;
    }
};

// Who does what.  Every workgroup finds out by itself: a launch before would
// cost more than that.  Threads take neighbouring requests (one, mostly).  The
// first workgroup writes down what the join needs to know.
template <int NA, int NB>
__device__ inline Shares shared_plan(const AttnArgs& a, const SharedArgs& s, uint32_t* tab, SharedGroup* grp,
                                     int* scratch, Start* start, int h, int x, int tid) {
    constexpr int W = kAttnWaves, rowsA = 16 * NA, rowsB = 16 * NB;
    int *longest = scratch + W, *tiles_all = longest + 1;
    Codebook book;
    book.load(a, h, tid);
    const int per = (a.B + kAttnThreads - 1) / kAttnThreads, b0 = tid * per;
    Rows mine_rw{};
    if (b0 < a.B) request_lens(a, b0, mine_rw);
    auto rows_of = [&](int b) {
        Rows rw = mine_rw;
        if (b != b0) request_lens(a, b, rw);
        return rw;
    };
    if (tid == 0) {
        *longest = 1;
        *tiles_all = 0;
    }
    for (int g = tid; g < s.groups; g += kAttnThreads) {
        int r0 = s.cu_groups[g], r1 = s.cu_groups[g + 1], p = s.prefix[g];
        const bool down = r1 < r0;
        r0 = r0 < 0 ? 0 : r0 > a.B ? a.B : r0;
        r1 = r1 < r0 ? r0 : r1 > a.B ? a.B : r1;
        p = p < 0 ? 0 : p > a.cap ? a.cap : p;
        SharedGroup y{};
        y.req0 = r0;
        y.req1 = r1;
        if (r1 > r0) {
            const int T = (int)a.T, c0 = a.cu[r0], c1 = a.cu[r1];
            const int t0 = c0 < 0 ? 0 : c0 > T ? T : c0, t1 = c1 < t0 ? t0 : c1 > T ? T : c1;
            y.tok0 = t0;
            y.rows = (t1 - t0) * a.G;  // <= 2^24
        }
        // one request shares with nobody; groups that descend: -1, see below
        y.blocks = down ? -1 : y.rows > 0 && r1 - r0 > 1 ? p / kKvBlock : 0;
        y.lo = 0x7fffffff;
        grp[g] = y;
    }
    book.build(tab, tid);
    __syncthreads();
    {
        // more tiles than there is room for: cu_groups or cu_q do not ascend
        int n = 0;
        for (int g = tid; g < s.groups; g += kAttnThreads) {
            const int y = grp[g].blocks < 0 ? s.wgs : grp[g].blocks ? (grp[g].rows + rowsA - 1) / rowsA : 0;
            n = n + y < s.wgs ? n + y : s.wgs;
        }
        if (n) atomicAdd(tiles_all, n);  // at most 256 wgs <= 2^31
    }
    __syncthreads();
    if (*tiles_all >= s.wgs) {
        for (int g = tid; g < s.groups; g += kAttnThreads) grp[g].blocks = 0;
        __syncthreads();
    }
    // what the query tokens see of the prefix, and their requests' own blocks
    int mine = 0, my_group = -1;
    for (int b = b0; b < b0 + per && b < a.B; ++b) {
        Rows rw = rows_of(b);
        const int g = group_of(grp, s.groups, b);
        if (b == b0) my_group = g;
        const int prefix = g >= 0 ? grp[g].blocks : 0;
        for (int rt = 0; rt < a.row_tiles; ++rt) {
            const Span sp = own_span(a, rw, rt, rowsB, prefix);
            mine += sp.hi > sp.lo ? sp.hi - sp.lo + kUnitBlocks : 0;
        }
        const int n = rw.qlen < a.max_q ? rw.qlen : a.max_q, end = prefix * kKvBlock;
        if (g < 0 || rw.qlen <= 0) continue;
        int lo, hi, first_hi, last_lo;
        bounds(a, rw, 0, lo, first_hi);  // both grow with the token
        bounds(a, rw, n - 1, last_lo, hi);
        hi = hi < end ? hi : end;
        if (hi > lo) {
            atomicMin(&grp[g].lo, lo);
            atomicMax(&grp[g].len, hi);
        }
        if (n < rw.qlen || last_lo > 0 || first_hi < end) grp[g].mixed = 1;
    }
    int total;
    int at = group_scan<W>(mine, scratch, total, tid) - mine;
    if (tid == 0) *tiles_all = 0;
    __syncthreads();
    for (int g = tid; g < s.groups; g += kAttnThreads) {
        SharedGroup& y = grp[g];
        const int lo = y.lo, hi = y.len;
        y.lo = hi > lo ? lo / kKvBlock : 0;
        y.len = hi > lo ? (hi + kKvBlock - 1) / kKvBlock - y.lo : 0;
        if (y.len > 0) {
            atomicAdd(tiles_all, (y.rows + rowsA - 1) / rowsA);
            atomicMax(longest, y.len);
        }
    }
    __syncthreads();
    // The least number k of blocks that every wave of a segment takes, with shares
    // that last as long, for which the workgroups are enough.  Where segments are
    // over before that because their groups are, their waves take shares as well.
    auto share_of = [&](int k) {
        const int y = (k * kBlockTime<NA> + kSegmentTime - kShareTime) / kOwnTime<NB>;
        return y > a.least ? y : a.least;
    };
    const int tiles = *tiles_all, whole = (*longest + W - 1) / W;
    auto extra_of = [&](int k) {
        const int y = k > whole ? ((k - whole) * kBlockTime<NA> - kAgainTime) / kOwnTime<NB> : 0;
        return y < a.least ? 0 : y;
    };
    int lo = 1, hi = whole;
    {
        const int room = W * (s.wgs - tiles), need = total / room + 2;
        const int k = need / kBlockTime<NA> * kOwnTime<NB> + kOwnTime<NB> + 1;
        hi = k > hi ? k : hi;  // enough: a segment a tile, and such shares
    }
    while (hi > lo) {
        const int step = (hi - lo + kAttnThreads - 1) / kAttnThreads, k = lo + tid * step;
        bool enough = false;
        if (k < hi) {
            // segments, at least their ceilings: lengths are below 2^22
            const float each = 1.000001f / (float)(k * W);
            int n = 0;
            for (int g = 0; g < s.groups && n <= s.wgs; ++g) {
                const int len = grp[g].len;
                const int64_t t = (int64_t)((grp[g].rows + rowsA - 1) / rowsA) * ((int)((float)(len - 1) * each) + 1);
                if (len > 0) n = t < s.wgs ? n + (int)t : s.wgs + 1;
            }
            enough = n <= s.wgs && (int64_t)(s.wgs - n) * W * share_of(k) + (int64_t)n * W * extra_of(k) >= total;
        }
        const uint64_t m = __ballot(enough);
        if ((tid & 63) == 0) scratch[tid >> 6] = m ? lo + (tid + __builtin_ctzll(m)) * step : hi;
        __syncthreads();
        int first = scratch[0];
#pragma unroll
        for (int w = 1; w < W; ++w) first = scratch[w] < first ? scratch[w] : first;
        __syncthreads();
        lo = first - lo >= step ? first - step + 1 : lo;
        hi = first;
    }
    Shares r;
    r.total = total;
    r.seg_len = hi * W;
    r.share = share_of(hi);
    r.extra = extra_of(hi);
    const int per_g = (s.groups + kAttnThreads - 1) / kAttnThreads, g0 = tid * per_g;
    int segs = 0;
    for (int g = g0; g < g0 + per_g && g < s.groups; ++g)
        segs += (grp[g].rows + rowsA - 1) / rowsA * ((grp[g].len + r.seg_len - 1) / r.seg_len);
    int base = group_scan<W>(segs, scratch, r.segments, tid) - segs;
    for (int g = g0; g < g0 + per_g && g < s.groups; ++g) {
        grp[g].base = base;
        base += (grp[g].rows + rowsA - 1) / rowsA * ((grp[g].len + r.seg_len - 1) / r.seg_len);
    }
    __syncthreads();
    const bool tell = x == 0 && h == 0;
    r.border = (s.wgs - r.segments) * W;
    const int w0 = (s.wgs - 1 - x) * W;
    const int64_t begin = r.begin(w0), stop = r.begin(w0 + W);
    if (tell && tid == 0) {
        s.head[0] = r.share;
        s.head[1] = r.extra;
        s.head[2] = r.border;
    }
    if (tell || (at < stop && at + mine > begin)) {
        for (int b = b0; b < b0 + per && b < a.B; ++b) {
            Rows rw = rows_of(b);
            const int g = b == b0 ? my_group : group_of(grp, s.groups, b);
            SharedGroup y{};
            if (g >= 0) y = grp[g];
            for (int rt = 0; rt < a.row_tiles; ++rt) {
                const Span sp = own_span(a, rw, rt, rowsB, y.blocks);
                const int unit = b * a.row_tiles + rt, n = sp.hi - sp.lo;
                if (tell) {
                    int4* u = s.unit + 3 * (int64_t)unit;
                    // the unit's rows among its group's; they are there unless cu_q descends
                    const int in = (rw.tok0 - y.tok0) * a.G + rw.r0;
                    const bool there = g >= 0 && in >= 0 && in + rw.n <= y.rows;
                    u[0] = make_int4(rw.tok0, rw.qlen, rw.seq, g);
                    u[1] = make_int4(at + kUnitBlocks, n, 0, 0);
                    u[2] = make_int4(there ? in : 0, y.base, there ? (y.len + r.seg_len - 1) / r.seg_len : 0, 0);
                }
                if (n <= 0) continue;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const int64_t from = r.begin(w0 + w);
                    if (from >= at && from < (int64_t)at + n + kUnitBlocks) start[w] = {unit, at};
                }
                at += n + kUnitBlocks;
            }
        }
    }
    __syncthreads();
    return r;
}

// Walk with DEPTH blocks on their way.  Two waves a SIMD, as many as the tiles'
// registers leave, do not cover the way to memory with one block each; a wave of
// few rows has the registers for more.  The pages of 64 blocks are looked up at
// once, one a lane: a lookup a block, which the compiler moves down to where its
// page is used, made every block wait for all loads before it.
template <int D, int DEPTH>
struct DeepWalk {
    const int32_t* table;
    int h, first, end, stride;
    int pages, later;  // of blocks 64 n + lane from the first, and the 64 behind them
    Block<D> blk[DEPTH];

    __device__ inline int lookup_pages(const AttnArgs& a, int n, int lane) const {
        // (a walk has fewer than 2^26 blocks)
        int b = first + (n + lane) * stride;
        b = b < end ? b : end - 1;
        return table[a.bpp == 1 ? b : (int)(((uint64_t)(uint32_t)b * a.bpp_magic) >> 32)];
    }
    __device__ inline Source source(const AttnArgs& a, int page, int b, int lane) const {
        const int in = a.bpp == 1 ? 0 : b - (int)(((uint64_t)(uint32_t)b * a.bpp_magic) >> 32) * (int)a.bpp;
        Source s;
        s.there = (uint32_t)page < (uint32_t)a.pages;
        const int64_t at = ((int64_t)(s.there ? page : 0) * a.Hkv + h) * 2;
        const int64_t code = (at * a.bpp + in) * (16 * D), row = at * a.page_size + in * kKvBlock;
        s.k = a.codes + code + lane * 16;
        s.v = a.codes + (code + (int64_t)a.bpp * (16 * D)) + lane * 16;
        s.ks = a.scales + row + 8 * (lane >> 4);
        s.vs = a.scales + (row + a.page_size) + 8 * (lane >> 4);
        return s;
    }
    // Block n of the walk (n - DEPTH is the one at hand).
    __device__ inline Source nth(const AttnArgs& a, int n, int lane) {
        int b = first + n * stride;
        b = b < end ? b : end - 1;
        return source(a, __builtin_amdgcn_readlane(pages, n & 63), b, lane);
    }
    __device__ inline void begin(const AttnArgs& a, const int32_t* row, int head, int lo, int hi, int by,
                                 int lane) {
        table = row;
        h = head;
        first = lo;
        end = hi;
        stride = by;
        pages = lookup_pages(a, 0, lane);
        later = (hi - lo) / 64 >= by ? lookup_pages(a, 64, lane) : pages;
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
            const Source src = nth(a, i, lane);
            blk[i].load_k(src);
            blk[i].load_v(src);
            // in this order: a first block loaded last would have the loop wait for all
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    template <int DT, int NT>
    __device__ inline void run(const AttnArgs& a, Wave<D, DT, NT>& wv, int lane) {
        const uint32_t lane4 = 4 * (lane & 31);
        const int g = lane >> 4;
        int n = 0;
        for (int b = first; b < end;) {
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) {
                if (b < end) {
                    if (((n + DEPTH) & 63) == 0) {  // the next 64 pages
                        pages = later;
                        later = lookup_pages(a, n + DEPTH + 64, lane);
                    }
                    const Source next = nth(a, n + DEPTH, lane);
                    wv.step(blk[i], next, b * kKvBlock, lane4, g, a.qk);
                }
                b += stride;
                ++n;
            }
        }
    }
};
template <int D, int NT>
constexpr int kDepth = NT > 2 ? 1 : NT == 1 && D <= 128 ? 3 : 2;

// Adds up the waves of a workgroup, and stores the rows' sums.  ml: [16 NT][W].
template <int D, int DT, int NT>
__device__ inline void store_segment(const AttnArgs& a, const Wave<D, DT, NT>& wv, int n, float* po,
                                     float* pml, uint32_t* tab, float2* ml, int wave, int lane) {
    constexpr int W = kAttnWaves;
    const int c = lane & 15, tid = wave * 64 + lane;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float l = wv.l[t];
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (lane < 16) ml[(t * 16 + c) * W + wave] = make_float2(wv.m[t], l);
    }
    __syncthreads();  // and nobody needs the table any more
    floatx4* buf = reinterpret_cast<floatx4*>(tab);  // [W][D / 16][64]: accumulators of a wave
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float top = kNoMax;
#pragma unroll
        for (int w = 0; w < W; ++w) top = fmaxf(top, ml[(t * 16 + c) * W + w].x);
        const float f = __builtin_amdgcn_exp2f(wv.m[t] - top);
#pragma unroll
        for (int p = 0; p < D / 16; ++p) {
            const int e = p / (D / 64), k = p % (D / 64);
            floatx4 x;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = wv.o[t][4 * k + j][e] * f;
            buf[(wave * (D / 16) + p) * 64 + lane] = x;
        }
        __syncthreads();
        for (int i = tid; i < 4 * D; i += 64 * W) {
            const int p = i >> 6, e = p / (D / 64), k = p % (D / 64), row = t * 16 + (i & 15);
            if (row >= n) continue;
            floatx4 x = buf[i];
#pragma unroll
            for (int w = 1; w < W; ++w) x += buf[w * 4 * D + i];
            const int d = (4 * ((i >> 4) & 3) + e) * (D / 16) + 4 * k;
            *reinterpret_cast<floatx4*>(po + row * D + d) = x;
            if (d == 0) {
                float most = kNoMax, sum = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) most = fmaxf(most, ml[row * W + w].x);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float2 y = ml[row * W + w];
                    sum += y.y * __builtin_amdgcn_exp2f(y.x - most);
                }
                *reinterpret_cast<float2*>(pml + row * 2) = make_float2(most, sum);
            }
        }
        if (t + 1 < NT) __syncthreads();
    }
}

// Grid (workgroups of a head, heads).
template <int D, int DT, int NA, int NB>
__global__ __launch_bounds__(kAttnThreads, 2) void k_kv4_shared_walk(AttnArgs a, SharedArgs s) {
    constexpr int W = kAttnWaves;
    extern __shared__ uint32_t tab[];
    float2* ml = reinterpret_cast<float2*>(tab + kTabBytes / 4);  // [16 NA][W]
    int* scratch = reinterpret_cast<int*>(ml + 16 * NA * W);
    Start* start = reinterpret_cast<Start*>(scratch + 8);
    SharedGroup* grp = reinterpret_cast<SharedGroup*>(start + W);
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = blockIdx.y, x = blockIdx.x;
    const Shares plan = shared_plan<NA, NB>(a, s, tab, grp, scratch, start, h, x, tid);
    if (x < plan.segments) {
        int g = 0, end = s.groups;  // the last group with base <= x: those without segments have the next one's
        while (end - g > 1) {
            const int mid = (g + end) / 2;
            if (grp[mid].base <= x) g = mid;
            else end = mid;
        }
        const SharedGroup y = grp[__builtin_amdgcn_readfirstlane(g)];
        const int segs = (y.len + plan.seg_len - 1) / plan.seg_len;
        const int k = x - y.base, tile = k / segs, seg = k - tile * segs;
        Rows rw;
        rw.tok0 = __builtin_amdgcn_readfirstlane(y.tok0);
        rw.qlen = 0;
        rw.seq = 0;
        rw.r0 = __builtin_amdgcn_readfirstlane(tile * 16 * NA);
        const int left = __builtin_amdgcn_readfirstlane(y.rows) - rw.r0;
        rw.n = left < 16 * NA ? left : 16 * NA;
        const int each = y.len / segs, rest = y.len - each * segs;  // the first `rest` have one more
        const int from = __builtin_amdgcn_readfirstlane(y.lo + seg * each + (seg < rest ? seg : rest));
        const int to = __builtin_amdgcn_readfirstlane(from + each + (seg < rest ? 1 : 0));
        const bool some = from + wave < to;
        typename Wave<D, DT, NA>::Raw raw;
        Wave<D, DT, NA>::fetch(a, rw, h, lane, raw);
        DeepWalk<D, kDepth<D, NA>> wk;
        if (some)
            wk.begin(a, a.table + __builtin_amdgcn_readfirstlane(y.req0) * a.max_pages, h, from + wave, to,
                     W, lane);
        // the positions of the prefix that each row's request lets it see
        const bool mixed = __builtin_amdgcn_readfirstlane(y.mixed);
        int2 seen[NA];
#pragma unroll
        for (int t = 0; t < NA; ++t) {
            seen[t] = make_int2(0, t * 16 + c < rw.n ? y.blocks * kKvBlock : 0);
            if (!mixed || t * 16 + c >= rw.n) continue;
            seen[t].y = 0;
            const int tok = rw.tok0 + divide(rw.r0 + t * 16 + c, a.G, a.G_magic);
            int b = y.req0, e = y.req1;  // the last request that does not begin behind the token
            while (e - b > 1) {
                const int mid = (b + e) / 2;
                if (a.cu[mid] <= tok) b = mid;
                else e = mid;
            }
            Rows its;
            request_lens(a, b, its);
            const int i = tok - its.tok0, end = y.blocks * kKvBlock;
            if (i < 0 || i >= its.qlen || i >= a.max_q) continue;
            bounds(a, its, i, seen[t].x, seen[t].y);
            seen[t].y = seen[t].y < end ? seen[t].y : end;
            if (seen[t].y <= seen[t].x) seen[t] = make_int2(0, 0);
        }
        Wave<D, DT, NA> wv;
        wv.init(a, rw, raw, lane);
        // the rows are those of several requests: each sees what its own does
        int lo = 0, hi = 0x7fffffff;
#pragma unroll
        for (int t = 0; t < NA; ++t) {
            wv.lo[t] = seen[t].x;
            wv.hi[t] = seen[t].y;
            if (t * 16 + c < rw.n) {
                lo = seen[t].x > lo ? seen[t].x : lo;
                hi = seen[t].y < hi ? seen[t].y : hi;
            }
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            const int y = __shfl_xor(lo, o), z = __shfl_xor(hi, o);
            lo = y > lo ? y : lo;
            hi = z < hi ? z : hi;
        }
        wv.inner_lo = __builtin_amdgcn_readfirstlane(lo);
        wv.inner_hi = __builtin_amdgcn_readfirstlane(hi);
        if (some) wk.run(a, wv, lane);
        const int64_t row = ((int64_t)h * s.wgs + x) * (16 * NA);
        store_segment<D, DT, NA>(a, wv, rw.n, a.part_o + row * D, a.part_ml + row * 2, tab, ml, wave, lane);
        if (plan.begin((s.wgs - 1 - x) * W) >= plan.total) return;
        Codebook book;
        book.load(a, h, tid);
        __syncthreads();  // sums of the segment lay in the table's place
        book.build(tab, tid);
        __syncthreads();
    }
    const int w = (s.wgs - 1 - x) * W + wave;
    const int64_t begin = plan.begin(w), to = plan.begin(w + 1), stop = to < plan.total ? to : plan.total;
    if (begin >= stop) return;
    const int units = a.B * a.row_tiles;
    const int64_t slots = (int64_t)h * (units + 2 * s.wgs * W);
    int unit = __builtin_amdgcn_readfirstlane(start[wave].unit);
    int64_t at = __builtin_amdgcn_readfirstlane(start[wave].at);
    int b = unit / a.row_tiles, rt = unit - b * a.row_tiles;
    Rows next;
    request_lens(a, b, next);
    while (at < stop && unit < units) {
        Rows rw = next;
        const int now = unit++, its = b, tile = rt;
        if (++rt == a.row_tiles) {
            rt = 0;
            if (++b < a.B) request_lens(a, b, next);  // on its way while this one is walked
        }
        const int g = __builtin_amdgcn_readfirstlane(group_of(grp, s.groups, its));
        const int prefix = g >= 0 ? __builtin_amdgcn_readfirstlane(grp[g].blocks) : 0;
        const Span sp = own_span(a, rw, tile, 16 * NB, prefix);
        const int all = sp.hi - sp.lo;
        if (all <= 0) continue;
        const int64_t first = at + kUnitBlocks;
        at = first + all;
        const int skip = begin > first ? (int)(begin - first) : 0;
        const int take = at < stop ? all - skip : (int)(stop - first) - skip;
        if (take <= 0) continue;
        typename Wave<D, DT, NB>::Raw raw;
        Wave<D, DT, NB>::fetch(a, rw, h, lane, raw);
        DeepWalk<D, kDepth<D, NB>> wk;
        wk.begin(a, a.table + its * a.max_pages, h, sp.lo + skip, sp.lo + skip + take, 1, lane);
        Wave<D, DT, NB> wv;
        wv.init(a, rw, raw, lane);
        wk.run(a, wv, lane);
        if (take == all && g < 0) {
            finish<D, DT, NB>(a, wv, rw, h, lane);
        } else {
            // one that lies whole in a share has a place of its own; the unit that a
            // share begins within has its place 0, one that goes on in the next
            // share its place 1
            const int64_t slot = take == all ? now : units + 2 * w + (first > begin);
            AttnArgs own = a;
            own.part_o = s.own_o;
            own.part_ml = s.own_ml;
            store_part<D, DT, NB>(own, wv, rw, slots + slot, lane);
        }
    }
}

// Grid (B, row tiles x heads, z): a workgroup takes every z-th row, join_rows of
// them at once; the threads of a row are D/4 wide, four dimensions each, and
// take every n-th of the row's sums: the prefix's segments, then the shares.
template <int D, int DT, int NA, int NB>
__global__ __launch_bounds__(kAttnThreads) void k_kv4_shared_join(AttnArgs a, SharedArgs s) {
    constexpr int kGroups = kAttnThreads / (D / 4);
    __shared__ floatx4 so[kAttnThreads];
    __shared__ float sm[kGroups], sl[kGroups];
    const int b = blockIdx.x;
    const int h = blockIdx.y / a.row_tiles, rt = blockIdx.y - h * a.row_tiles;
    const int unit = b * a.row_tiles + rt, units = a.B * a.row_tiles;
    const int4 u0 = s.unit[3 * (int64_t)unit], u1 = s.unit[3 * (int64_t)unit + 1], u2 = s.unit[3 * (int64_t)unit + 2];
    Shares plan{};
    plan.share = s.head[0];
    plan.extra = s.head[1];
    plan.border = s.head[2];
    const int64_t lo = u1.x, hi = lo + u1.y;
    const int w0 = hi > lo ? plan.wave_of(lo) : 0, w1 = hi > lo ? plan.wave_of(hi - 1) : 0;
    const bool whole = hi > lo && w0 == w1;
    if (whole && u0.w < 0) return;
    Rows rw;
    rw.tok0 = u0.x;
    rw.qlen = u0.y;
    rw.seq = u0.z;
    tile_rows(a, rw, rt * 16 * NB, 16 * NB);
    const int segs = u2.z, own = hi > lo ? w1 - w0 + 1 : 0, all = segs + own;
    const int64_t slots = (int64_t)h * (units + 2 * s.wgs * kAttnWaves);
    const int tid = threadIdx.x, grp_no = tid / (D / 4), d = 4 * (tid % (D / 4));
    const int n = kGroups / a.join_rows, sub = grp_no % n;  // threads of a row, which of them
    for (int r0 = 0; r0 * (int)gridDim.z < rw.n; r0 += a.join_rows) {
        const int row = (r0 + grp_no / n) * gridDim.z + blockIdx.z;
        // the row's place in its group's tiles
        const int in = u2.x + row, tile = in / (16 * NA);
        const int64_t first = ((int64_t)h * s.wgs + u2.y + tile * segs) * (16 * NA) + (in - tile * 16 * NA);
        float top = kNoMax, sum = 0.f;
        floatx4 o = {0, 0, 0, 0};
        if (row < rw.n) {
            constexpr int kBatch = 4;  // sums loaded at a time
            for (int w = sub; w < all; w += kBatch * n) {
                float2 ml[kBatch];
                floatx4 y[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int x = w + i * n < all ? w + i * n : w;
                    const float *po = a.part_o, *pm = a.part_ml;
                    int64_t at;
                    if (x < segs) {
                        at = first + (int64_t)x * (16 * NA);
                    } else {
                        const int v = w0 + x - segs;
                        po = s.own_o;
                        pm = s.own_ml;
                        at = (slots + (whole ? unit : units + 2 * v + (v == w0 && lo > plan.begin(v) ? 1 : 0))) *
                                 a.part_rows + row;
                    }
                    ml[i] = *reinterpret_cast<const float2*>(pm + at * 2);
                    y[i] = *reinterpret_cast<const floatx4*>(po + at * D + d);
                }
                float nm = top;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) nm = fmaxf(nm, ml[i].x);
                float f = __builtin_amdgcn_exp2f(top - nm);
                o *= f;
                sum *= f;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    f = w + i * n < all ? __builtin_amdgcn_exp2f(ml[i].x - nm) : 0.f;
                    o += y[i] * f;
                    sum += ml[i].y * f;
                }
                top = nm;
            }
        }
        if (n > 1) {
            so[tid] = o;
            if (d == 0) {
                sm[grp_no] = top;
                sl[grp_no] = sum;
            }
            __syncthreads();
            if (sub == 0) {
                float most = top;
                for (int i = 1; i < n; ++i) most = fmaxf(most, sm[grp_no + i]);
                float f = __builtin_amdgcn_exp2f(top - most);
                sum *= f;
                o *= f;
                for (int i = 1; i < n; ++i) {
                    f = __builtin_amdgcn_exp2f(sm[grp_no + i] - most);
                    sum += sl[grp_no + i] * f;
                    o += so[tid + i * (D / 4)] * f;
                }
                top = most;
            }
            __syncthreads();
        }
        if (sub == 0 && row < rw.n) {
            const int r = rw.r0 + row, i = divide(r, a.G, a.G_magic), head = h * a.G + r - i * a.G;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            store_out<DT>(a, rw.tok0 + i, head, D, d, o * inv);
            if (a.lse && d == 0)
                a.lse[(int64_t)(rw.tok0 + i) * a.Hq + head] =
                    (top + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
        }
    }
}

template <int D, int DT, int NA, int NB>
hipError_t shared_run(const AttnArgs& a, const SharedArgs& s, const SharedPlan& p, hipStream_t st) {
    static LdsAttr rec;
    auto walk = k_kv4_shared_walk<D, DT, NA, NB>;
    constexpr int fixed = kTabBytes + 16 * NA * kAttnWaves * 8 + 32 + kAttnWaves * sizeof(Start);
    static_assert(fixed + kSharedGroups * sizeof(SharedGroup) <= 80 * 1024, "two workgroups a CU");
    hipError_t e = ensure_lds(rec, reinterpret_cast<const void*>(walk), 80 * 1024);
    if (e != hipSuccess) return e;
    walk<<<dim3((unsigned)s.wgs, (unsigned)a.Hkv), dim3(kAttnThreads),
           fixed + s.groups * sizeof(SharedGroup), st>>>(a, s);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_kv4_shared_join<D, DT, NA, NB>
        <<<dim3((unsigned)a.B, (unsigned)(a.Hkv * a.row_tiles), (unsigned)p.join_z), dim3(kAttnThreads), 0,
           st>>>(a, s);
    return hipGetLastError();
}

template <int D, int DT>
hipError_t shared_cols(const AttnArgs& a, const SharedArgs& s, const SharedPlan& p, hipStream_t st) {
    if constexpr (kTileCols<D> > 1) {
        if (p.col_blocks > 1) return shared_run<D, DT, 3, 2>(a, s, p, st);
        if (p.group_cols == 3) return shared_run<D, DT, 3, 1>(a, s, p, st);
        if (p.group_cols == 2) return shared_run<D, DT, 2, 1>(a, s, p, st);
    }
    return shared_run<D, DT, 1, 1>(a, s, p, st);
}

template <int D>
hipError_t shared_d(const AttnArgs& a, const SharedArgs& s, const SharedPlan& p, int dtype,
                    hipStream_t st) {
    return dtype == FK_BF16 ? shared_cols<D, FK_BF16>(a, s, p, st) : shared_cols<D, FK_F16>(a, s, p, st);
}

}  // namespace
}  // namespace fk
