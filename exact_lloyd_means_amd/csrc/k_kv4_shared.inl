// k_kv4_shared.inl -- attention of requests that share a prefix
// (fk_kv4_attention_shared), on the waves of k_kv4_attn.inl.
//
// The query rows of a group's requests lie one after another, so 16 NA of them
// make a tile that walks the prefix once, whatever requests they belong to: for
// single tokens a tile serves 16 NA / G requests instead of one, and a block's
// codes are read and looked up that many times less.  What lies behind the
// prefix is walked for each request as in the split form.  Three launches:
//
//   k_kv4_shared_plan  one workgroup: what every query token sees of the prefix,
//                      the segments of the tiles' keys (one a workgroup), the
//                      shares of the requests' own keys (one a wave)
//   k_kv4_shared_walk  segments and shares; sums of rows go to the workspace
//   k_kv4_shared_join  adds up the segments and shares of each request, in order
//
// Both kinds of work run in one launch; the plan gives each as many workgroups as
// let them end together.
#pragma once

#include "k_kv4_attn.inl"
#include "serve_internal.h"

namespace fk {
namespace {

constexpr int kPlanWaves = 16;  // at most

// What balances the two kinds of work, in tenths of a microsecond at two waves a
// SIMD with heads of 128: a block of 16 NT rows; what a segment costs beside its
// blocks (codes on their way, waves added up); a unit of a share likewise, in
// blocks of its own.
template <int NT>
constexpr int kBlockTime = 3 + 5 * NT;
template <int NT>
constexpr int kOwnTime = NT < 2 ? 13 : kBlockTime<NT>;
constexpr int kSegmentTime = 110, kShareTime = 80;
constexpr int kUnitBlocks = kSharedUnit;

// Row tiles of requests.
__device__ inline Span own_span(const AttnArgs& a, Rows& rw, int rt, int rows, int prefix) {
    Span sp = tile_rows(a, rw, rt * rows, rows);
    sp.lo = sp.lo > prefix ? sp.lo : prefix;
    sp.hi = sp.hi > sp.lo ? sp.hi : sp.lo;
    return sp;
}

// Inclusive scan over a workgroup of up to kPlanWaves waves.
__device__ inline int64_t plan_scan(int64_t x, int64_t* scratch, int64_t& total, int tid) {
    const int lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t y = __shfl_up((long long)x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // scratch may still be read
    if (lane == 63) scratch[wave] = x;
    __syncthreads();
    total = 0;
    for (int w = 0; w < waves; ++w) {
        const int64_t y = scratch[w];
        if (w < wave) x += y;
        total += y;
    }
    return x;
}

struct SharedGroup {  // in LDS
    int req0, req1;   // its requests
    int tok0, tok1;   // their query tokens
    int blocks;       // of the prefix
    int least, most;  // first and one past the last position that a row sees
    int tiles, lo, len, segs, base;
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
    return groups > 0 && b >= g[lo].req0 && b < g[lo].req1 ? lo : -1;
}

// A thread takes neighbouring requests (one, mostly) and groups.
template <int NA, int NB>
__global__ __launch_bounds__(64 * kPlanWaves) void k_kv4_shared_plan(AttnArgs a, SharedArgs s) {
    extern __shared__ SharedGroup grp[];
    __shared__ int64_t scratch[kPlanWaves];
    __shared__ int longest, best;
    const int tid = threadIdx.x, threads = blockDim.x;
    constexpr int rowsA = 16 * NA, rowsB = 16 * NB;
    const int per = (a.B + threads - 1) / threads, b0 = tid * per;
    Rows mine_rw{};
    if (b0 < a.B) request_lens(a, b0, mine_rw);
    auto rows_of = [&](int b) {
        Rows rw = mine_rw;
        if (b != b0) request_lens(a, b, rw);
        return rw;
    };
    int64_t bound = 0, total;  // tiles; beyond what there is room for if lists descend
    if (tid == 0) longest = 1;
    for (int g = tid; g < s.groups; g += threads) {
        int r0 = s.cu_groups[g], r1 = s.cu_groups[g + 1], p = s.prefix[g];
        if (r1 < r0) bound += s.wgs;
        r0 = r0 < 0 ? 0 : r0 > a.B ? a.B : r0;
        r1 = r1 < r0 ? r0 : r1 > a.B ? a.B : r1;
        p = p < 0 ? 0 : p > a.cap ? a.cap : p;
        SharedGroup x{};
        x.req0 = r0;
        x.req1 = r1;
        if (r1 > r0) {
            const int T = (int)a.T, t0 = a.cu[r0], t1 = a.cu[r1];
            x.tok0 = t0 < 0 ? 0 : t0 > T ? T : t0;
            x.tok1 = t1 < x.tok0 ? x.tok0 : t1 > T ? T : t1;
        }
        x.blocks = p / kKvBlock;
        // rows that one tile of their own would hold share nothing
        const int64_t rows = (int64_t)(x.tok1 - x.tok0) * a.G;
        if (rows <= rowsB) x.blocks = 0;
        if (x.blocks) bound += (rows + rowsA - 1) / rowsA;
        x.least = 0x7fffffff;
        x.most = 0;
        grp[g] = x;
    }
    plan_scan(bound, scratch, total, tid);
    if (total >= s.wgs) {
        // cu_groups or cu_q do not ascend: nothing is shared
        for (int g = tid; g < s.groups; g += threads) grp[g].blocks = 0;
        __syncthreads();
    }
    // what the query tokens see of the prefix, and their requests' own blocks
    int64_t mine = 0;
    int my_group = -1;
    for (int b = b0; b < b0 + per && b < a.B; ++b) {
        Rows rw = rows_of(b);
        int g = group_of(grp, s.groups, b);
        if (g >= 0 && grp[g].blocks == 0) g = -1;
        s.req[b] = g;
        if (b == b0) my_group = g;
        const int prefix = g >= 0 ? grp[g].blocks : 0;
        for (int rt = 0; rt < a.row_tiles; ++rt) {
            const Span sp = own_span(a, rw, rt, rowsB, prefix);
            mine += sp.hi > sp.lo ? sp.hi - sp.lo + kUnitBlocks : 0;
        }
        if (g < 0) continue;
        const int end = prefix * kKvBlock, n = rw.qlen < a.max_q ? rw.qlen : a.max_q;
        int least = 0x7fffffff, most = 0;
        for (int i = 0; i < rw.qlen; ++i) {
            int lo = 0, hi = 0;
            if (i < n) {
                bounds(a, rw, i, lo, hi);
                hi = hi < end ? hi : end;
                if (hi > lo) {
                    least = lo < least ? lo : least;
                    most = hi > most ? hi : most;
                } else {
                    lo = hi = 0;
                }
            }
            s.seen[rw.tok0 + i] = make_int2(lo, hi);
        }
        atomicMin(&grp[g].least, least);
        atomicMax(&grp[g].most, most);
    }
    int64_t blocks;  // and kUnitBlocks for each unit
    int64_t at = plan_scan(mine, scratch, blocks, tid) - mine;
    int64_t tiles = 0;
    for (int g = tid; g < s.groups; g += threads) {
        SharedGroup& x = grp[g];
        x.lo = x.most > x.least ? x.least / kKvBlock : 0;
        x.len = x.most > x.least ? (x.most + kKvBlock - 1) / kKvBlock - x.lo : 0;
        x.tiles = x.len > 0 ? (int)(((int64_t)(x.tok1 - x.tok0) * a.G + rowsA - 1) / rowsA) : 0;
        tiles += x.tiles;
        atomicMax(&longest, x.len);
    }
    plan_scan(tiles, scratch, tiles, tid);
    // The least number k of blocks that every wave of a segment takes, with shares
    // that last as long, for which the workgroups are enough.
    constexpr int W = kAttnWaves;
    auto share_of = [&](int64_t k) {
        const int64_t x = (k * kBlockTime<NA> + kSegmentTime - kShareTime) / kOwnTime<NB>;
        return x > a.least ? x : a.least;
    };
    int64_t lo = 1, hi = (longest + W - 1) / W;
    {
        const int64_t need = (blocks + W * (s.wgs - tiles) - 1) / (W * (s.wgs - tiles));
        const int64_t k = (need + 1) * kOwnTime<NB> / kBlockTime<NA> + 1;
        hi = k > hi ? k : hi;  // enough: a segment a tile, and such shares
    }
    while (hi > lo) {
        const int64_t step = (hi - lo + threads - 1) / threads, x = lo + tid * step;
        if (tid == 0) best = (int)hi;
        __syncthreads();
        if (x < hi) {
            const int64_t each = W * share_of(x);
            int64_t n = (blocks + each - 1) / each;
            for (int g = 0; g < s.groups; ++g)
                if (grp[g].tiles) n += grp[g].tiles * ((grp[g].len + x * W - 1) / (x * W));
            if (n <= s.wgs) atomicMin(&best, (int)x);
        }
        __syncthreads();
        hi = best;
        __syncthreads();
        lo = hi - step + 1 > lo ? hi - step + 1 : lo;
    }
    const int len = (int)hi * W, share = (int)share_of(hi);
    const int per_g = (s.groups + threads - 1) / threads, g0 = tid * per_g;
    int64_t segs = 0, segments;
    for (int g = g0; g < g0 + per_g && g < s.groups; ++g)
        segs += (int64_t)grp[g].tiles * ((grp[g].len + len - 1) / len);
    int64_t base = plan_scan(segs, scratch, segments, tid) - segs;
    for (int g = g0; g < g0 + per_g && g < s.groups; ++g) {
        SharedGroup& x = grp[g];
        x.base = (int)base;
        x.segs = (x.len + len - 1) / len;
        base += (int64_t)x.tiles * x.segs;
        s.group[2 * g] = make_int4(x.tok0, x.base, x.segs, x.blocks);
        s.group[2 * g + 1] = make_int4((x.tok1 - x.tok0) * a.G, 0, 0, 0);
    }
    if (tid == 0) {
        s.head[0] = (int)segments;
        s.head[1] = (int)blocks;
        s.head[2] = share;
        a.prefix[a.B * a.row_tiles] = (int)blocks;
    }
    // where units and shares begin
    for (int b = b0; b < b0 + per && b < a.B; ++b) {
        Rows rw = rows_of(b);
        const int g = b == b0 ? my_group : s.req[b], prefix = g >= 0 ? grp[g].blocks : 0;
        for (int rt = 0; rt < a.row_tiles; ++rt) {
            const Span sp = own_span(a, rw, rt, rowsB, prefix);
            const int unit = b * a.row_tiles + rt, n = sp.hi > sp.lo ? sp.hi - sp.lo + kUnitBlocks : 0;
            a.prefix[unit] = (int)at;
            for (int64_t w = (at + share - 1) / share; w * share < at + n; ++w) s.start[w] = unit;
            at += n;
        }
    }
    __syncthreads();
    for (int i = tid; i < (int)segments; i += threads) {
        int l = 0, h = s.groups;  // the last group with base <= i: those without tiles have the next one's
        while (h - l > 1) {
            const int mid = (l + h) / 2;
            if (grp[mid].base <= i) l = mid;
            else h = mid;
        }
        const SharedGroup x = grp[l];
        const int k = i - x.base, tile = k / x.segs, seg = k - tile * x.segs;
        const int from = x.lo + seg * len, to = from + len < x.lo + x.len ? from + len : x.lo + x.len;
        s.segment[2 * i] = make_int4(x.req0, x.tok0, x.tok1 - x.tok0, tile);
        s.segment[2 * i + 1] = make_int4(from, to, 0, 0);
    }
}

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
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = blockIdx.y, segments = s.head[0];
    const int x = blockIdx.x;
    if (x < segments) {
        const int4 d0 = s.segment[2 * x], d1 = s.segment[2 * x + 1];
        Rows rw;
        rw.tok0 = __builtin_amdgcn_readfirstlane(d0.y);
        rw.qlen = __builtin_amdgcn_readfirstlane(d0.z);
        rw.seq = 0;
        rw.r0 = __builtin_amdgcn_readfirstlane(d0.w) * 16 * NA;
        const int left = rw.qlen * a.G - rw.r0;
        rw.n = left < 16 * NA ? left : 16 * NA;
        const int from = __builtin_amdgcn_readfirstlane(d1.x), to = __builtin_amdgcn_readfirstlane(d1.y);
        const bool some = from + wave < to;
        typename Wave<D, DT, NA>::Raw raw;
        Wave<D, DT, NA>::fetch(a, rw, h, lane, raw);
        Walk<D> wk;
        if (some)
            wk.begin(a, a.table + __builtin_amdgcn_readfirstlane(d0.x) * a.max_pages, h, from + wave, to,
                     W, lane);
        int2 seen[NA];
#pragma unroll
        for (int t = 0; t < NA; ++t) {
            const int r = rw.r0 + t * 16 + c;
            seen[t] = t * 16 + c < rw.n ? s.seen[rw.tok0 + divide(r, a.G, a.G_magic)] : make_int2(0, 0);
        }
        build_table(tab, a.codebook, a.Hkv, h, tid, kAttnThreads);
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
        __syncthreads();
        if (some) wk.run(a, wv, lane);
        const int64_t row = ((int64_t)h * s.wgs + x) * (16 * NA);
        store_segment<D, DT, NA>(a, wv, rw.n, a.part_o + row * D, a.part_ml + row * 2, tab, ml, wave, lane);
        return;
    }
    // shares of the line of units: each is kUnitBlocks without work, then its blocks
    const int total = s.head[1], share = s.head[2];
    const int w = (x - segments) * W + wave;
    if ((int64_t)(x - segments) * W * share >= total) return;
    int64_t at = (int64_t)w * share;
    const int64_t stop = at + share < total ? at + share : total;
    int unit = at < total ? __builtin_amdgcn_readfirstlane(s.start[w]) : 0;
    build_table(tab, a.codebook, a.Hkv, h, tid, kAttnThreads);
    __syncthreads();
    const int units = a.B * a.row_tiles;
    const int64_t slots = (int64_t)h * (units + 2 * s.wgs * W);
    for (; at < stop && unit < units; ++unit) {
        const int b = unit / a.row_tiles, rt = unit - b * a.row_tiles;
        Rows rw;
        request_lens(a, b, rw);
        const int g = s.req[b], prefix = g >= 0 ? s.group[2 * g].w : 0;
        const Span sp = own_span(a, rw, rt, 16 * NB, prefix);
        const int all = sp.hi - sp.lo;
        if (all <= 0) continue;
        const int64_t first = a.prefix[unit] + kUnitBlocks;
        const int skip = at > first ? (int)(at - first) : 0;
        const int take = first + all < stop ? all - skip : (int)(stop - first) - skip;
        if (take > 0) {
            typename Wave<D, DT, NB>::Raw raw;
            Wave<D, DT, NB>::fetch(a, rw, h, lane, raw);
            Walk<D> wk;
            wk.begin(a, a.table + b * a.max_pages, h, sp.lo + skip, sp.lo + skip + take, 1, lane);
            Wave<D, DT, NB> wv;
            wv.init(a, rw, raw, lane);
            wk.run(a, wv, lane);
            if (take == all && g < 0) {
                finish<D, DT, NB>(a, wv, rw, h, lane);
            } else {
                // one that lies whole in a share has a place of its own; a share's
                // first unit has place 0 of the share, one that begins in it 1
                const int64_t slot = take == all ? unit : units + 2 * w + (first > (int64_t)w * share);
                AttnArgs to = a;
                to.part_o = s.own_o;
                to.part_ml = s.own_ml;
                store_part<D, DT, NB>(to, wv, rw, slots + slot, lane);
            }
        }
        at = first + all;
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
    const int64_t lo = a.prefix[unit] + kUnitBlocks, hi = a.prefix[unit + 1];
    const int share = s.head[2], g = s.req[b];
    const int w0 = (int)(lo / share), w1 = hi > lo ? (int)((hi - 1) / share) : w0;
    const bool whole = hi > lo && w0 == w1;
    if (whole && g < 0) return;
    Rows rw;
    request_lens(a, b, rw);
    tile_rows(a, rw, rt * 16 * NB, 16 * NB);
    int4 grp = g >= 0 ? s.group[2 * g] : make_int4(0, 0, 0, 0);
    // the request's rows are among its group's unless cu_q descends
    const int64_t in0 = (int64_t)(rw.tok0 - grp.x) * a.G + rw.r0;
    if (g >= 0 && (in0 < 0 || in0 + rw.n > s.group[2 * g + 1].x)) grp.z = 0;
    const int own = hi > lo ? w1 - w0 + 1 : 0, all = grp.z + own;
    const int64_t slots = (int64_t)h * (units + 2 * s.wgs * kAttnWaves);
    const int tid = threadIdx.x, grp_no = tid / (D / 4), d = 4 * (tid % (D / 4));
    const int n = kGroups / a.join_rows, sub = grp_no % n;  // threads of a row, which of them
    for (int r0 = 0; r0 * (int)gridDim.z < rw.n; r0 += a.join_rows) {
        const int row = (r0 + grp_no / n) * gridDim.z + blockIdx.z;
        // the row's place in its group's tiles
        const int in = (int)in0 + row, tile = in / (16 * NA);
        const int64_t first = ((int64_t)h * s.wgs + grp.y + tile * grp.z) * (16 * NA) + (in - tile * 16 * NA);
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
                    if (x < grp.z) {
                        at = first + (int64_t)x * (16 * NA);
                    } else {
                        const int v = w0 + x - grp.z;
                        po = s.own_o;
                        pm = s.own_ml;
                        at = (slots + (whole ? unit : units + 2 * v + (v == w0 && lo > (int64_t)v * share ? 1 : 0))) *
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
    static LdsAttr rec, rec_plan;
    auto plan = k_kv4_shared_plan<NA, NB>;
    auto walk = k_kv4_shared_walk<D, DT, NA, NB>;
    constexpr int lds = kTabBytes + 16 * NA * kAttnWaves * 8;
    hipError_t e = ensure_lds(rec, reinterpret_cast<const void*>(walk), lds);
    if (e != hipSuccess) return e;
    e = ensure_lds(rec_plan, reinterpret_cast<const void*>(plan), kSharedGroups * sizeof(SharedGroup));
    if (e != hipSuccess) return e;
    const int threads = a.B <= 256 && s.groups <= 256 ? 256 : 64 * kPlanWaves;
    plan<<<dim3(1), dim3(threads), s.groups * sizeof(SharedGroup), st>>>(a, s);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    walk<<<dim3((unsigned)s.wgs, (unsigned)a.Hkv), dim3(kAttnThreads), lds, st>>>(a, s);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_kv4_shared_join<D, DT, NA, NB>
        <<<dim3((unsigned)a.B, (unsigned)(a.Hkv * a.row_tiles), (unsigned)p.join_z), dim3(kAttnThreads), 0,
           st>>>(a, s);
    return hipGetLastError();
}

template <int D, int DT>
hipError_t shared_cols(const AttnArgs& a, const SharedArgs& s, const SharedPlan& p, hipStream_t st) {
    constexpr int NA = kTileCols<D>;
    if constexpr (NA > 1)
        if (p.col_blocks > 1) return shared_run<D, DT, NA, NA>(a, s, p, st);
    return shared_run<D, DT, NA, 1>(a, s, p, st);
}

template <int D>
hipError_t shared_d(const AttnArgs& a, const SharedArgs& s, const SharedPlan& p, int dtype,
                    hipStream_t st) {
    return dtype == FK_BF16 ? shared_cols<D, FK_BF16>(a, s, p, st) : shared_cols<D, FK_F16>(a, s, p, st);
}

}  // namespace
}  // namespace fk
