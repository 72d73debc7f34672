// k_kv_pages.hip -- pages of the cache forked, returned, copied and compacted
// (fk_kv_fork, fk_kv_compact, fk_kv4_copy).
#include "serve_internal.h"

namespace fk {
namespace {

constexpr int kNone = 0x7fffffff;

// ---- fork ----------------------------------------------------------------------------
//
// Every pair is worked on by one wave, in five steps over all pairs, each of
// which needs the whole of the one before:
//   read   who the pair's row and source are, what it takes; entries of the
//          source put aside; counters of the pages that it touches cleared
//   count  per page: rows that give it up, that take it whole, the first that
//          goes on writing in it
//   sum    per pair: pages that nobody holds any more, whether it needs a copy
//   give   those pages to the list, in order
//   take   pages for the copies from the list; rows, lengths and shares written
// Sums are of integers and the order is that of the pairs, so timing shows
// nowhere.  Bound by the chain of dependent reads of the five steps; they are
// one launch where one workgroup will do (4 rows of 16 pages: 8.6 us), else five
// (240 rows of 64-121 pages: 3.4 to 5.6 us each).
//
// A wave finds the other pairs of its row, and what the pairs before it give up
// and copy, by reading all pairs.  That is n^2 in all, so many pairs have three
// launches more: names and least lengths by row (two), sums of the pairs before
// (one workgroup).  Rows that return their last pages, us with them / without: 1024
// 26 / 26, 2048 27 / 36, 16384 72 / 560, 65536 226 / 8440.
//
// Entries that a row holds and takes again at the same place (those before its
// new end when it is its own source, pages that it shares with its source) give
// and take the same page and are left out.

// Of info[i]; kFrom: entries before it are left out.
enum { kAct, kRow, kFrom, kLen, kHeld, kGone, kCopy, kEnd };

__device__ inline bool page_of(const ForkArgs& a, int p) { return p >= 0 && p < a.N; }
__device__ inline int held_of(const ForkArgs& a, int len) {
    const int64_t h = len <= 0 ? 0 : ((int64_t)len + a.P - 1) / a.P;
    return (int)(h < a.M ? h : a.M);
}
__device__ inline int row_len(const ForkArgs& a, int r) {
    const int64_t n = a.lens[r], most = a.M * a.P;
    return (int)(n < 0 ? 0 : n < most ? n : most);
}
__device__ inline int wave_min(int x) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const int y = __shfl_xor(x, o);
        x = y < x ? y : x;
    }
    return x;
}
__device__ inline int wave_add(int x) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
    return x;
}

// What atomics changed is read past the first cache, which they do not change.
template <typename T>
__device__ inline T changed(const T* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline void clear_page(const ForkArgs& a, int p) {
    a.count[p] = 0;
    a.tail[p] = kNone;
    a.first[p] = ~(uint64_t)0;
}

__device__ inline void fork_read(const ForkArgs& a, int i, int lane) {
    int* info = a.info + 8 * i;
    const int r = a.rows[i];
    int first = kNone, least = kNone;
    bool act = r >= 0 && r < a.R;
    if (act && a.named) {
        first = a.named[2 * (int64_t)r];
        least = a.named[2 * (int64_t)r + 1];
        act = first == i;
    } else if (act) {
        for (int j = lane; j < a.n; j += 64)
            if (a.rows[j] == r) {
                first = j < first ? j : first;
                least = a.keep[j] < least ? a.keep[j] : least;
            }
        first = wave_min(first);
        least = wave_min(least);
        act = first == i;
    }
    int s = -1, len = 0, held = 0;
    if (act) {
        const int now = row_len(a, r);
        s = a.sources ? a.sources[i] : r;
        s = s >= 0 && s < a.R ? s : -1;
        len = s >= 0 ? row_len(a, s) : 0;
        least = least < 0 ? 0 : least;
        len = least < len ? least : len;
        held = held_of(a, now);
        act = !(s == r && len == now);
    }
    const int from = s == r ? len / a.P : 0;
    if (lane == 0) {
        info[kAct] = act;
        info[kRow] = r;
        info[kFrom] = from;
        info[kLen] = len;
        info[kHeld] = held;
    }
    if (!act) return;
    const int end = held_of(a, len);
    for (int e = from + lane; e < held || e < end; e += 64) {
        const int old = e < held ? a.table[r * a.M + e] : -1, p = e < end ? a.table[s * a.M + e] : -1;
        if (e < end) a.fresh[i * a.M + e] = page_of(a, p) ? p : -1;
        if (page_of(a, old)) clear_page(a, old);
        if (page_of(a, p)) clear_page(a, p);
    }
}

__device__ inline uint64_t entry_no(int i, int e) { return (uint64_t)(uint32_t)i << 32 | (uint32_t)e; }

__device__ inline void fork_count(const ForkArgs& a, int i, int lane) {
    const int* info = a.info + 8 * i;
    if (!info[kAct]) return;
    const int* row = a.table + info[kRow] * a.M;
    const int* fresh = a.fresh + i * a.M;
    const int whole = info[kLen] / a.P, held = info[kHeld];
    for (int e = info[kFrom] + lane; e < held || e < whole; e += 64) {
        const int old = e < held ? row[e] : -1, p = e < whole ? fresh[e] : -1;
        if (old == p) continue;
        if (page_of(a, old)) {
            atomicAdd(&a.count[old], -1);
            atomicMin((unsigned long long*)&a.first[old], (unsigned long long)entry_no(i, e));
        }
        if (p >= 0) atomicAdd(&a.count[p], 1);
    }
    if (lane == 0 && info[kLen] % a.P && fresh[whole] >= 0) atomicMin(&a.tail[fresh[whole]], i);
}

// Rows that hold a page whole afterwards, not counting one that goes on in it.
__device__ inline int base_of(const ForkArgs& a, int p) { return a.shares[p] + 1 + changed(&a.count[p]); }
__device__ inline bool gives_up(const ForkArgs& a, int p, int i, int e) {
    return base_of(a, p) <= 0 && changed(&a.tail[p]) == kNone && changed(&a.first[p]) == entry_no(i, e);
}

__device__ inline void fork_sum(const ForkArgs& a, int i, int lane) {
    int* info = a.info + 8 * i;
    if (!info[kAct]) {
        if (lane == 0) info[kGone] = info[kCopy] = 0;
        return;
    }
    const int* row = a.table + info[kRow] * a.M;
    int gone = 0;
    for (int e = info[kFrom] + lane; e < info[kHeld]; e += 64) {
        const int p = row[e];
        if (page_of(a, p) && gives_up(a, p, i, e)) ++gone;
    }
    gone = wave_add(gone);
    if (lane) return;
    const int whole = info[kLen] / a.P;
    const int p = info[kLen] % a.P ? a.fresh[i * a.M + whole] : -1;
    const bool mine = p >= 0 && base_of(a, p) <= 0 && changed(&a.tail[p]) == i;
    info[kGone] = gone;
    info[kCopy] = p >= 0 && !mine;
    info[kEnd] = mine ? p : -1;  // the page that the row goes on in
}

__device__ inline int next_shares(const ForkArgs& a, int p) {
    const int base = base_of(a, p);
    const int refs = base > 0 ? base : changed(&a.tail[p]) != kNone;
    return refs > 1 ? refs - 1 : 0;
}

// Sums of one field over pairs [0, i) and over all.
__device__ inline void before(const ForkArgs& a, int field, int i, int lane, int& upto, int& all) {
    int x = 0, y = 0;
    for (int j = lane; j < a.n; j += 64) {
        const int v = a.info[8 * j + field];
        y += v;
        x += j < i ? v : 0;
    }
    upto = wave_add(x);
    all = wave_add(y);
}

__device__ inline int list_len(const ForkArgs& a) {
    const int n = *a.free_count;
    return n < 0 ? 0 : n > a.N ? (int)a.N : n;
}

// The list with the pages given up, and how many of it the copies take.
__device__ inline void count_list(const ForkArgs& a, int gone, int copies) {
    const int64_t have = (int64_t)list_len(a) + gone;
    a.have[0] = (int)(have < a.N ? have : a.N);
    a.have[1] = copies < a.have[0] ? copies : a.have[0];
}

__device__ inline void fork_give(const ForkArgs& a, int i, int lane) {
    const int* info = a.info + 8 * i;
    int upto, all;
    if (i == 0 && !a.upto) {
        int copies;
        before(a, kGone, 0, lane, upto, all);
        before(a, kCopy, 0, lane, upto, copies);
        if (lane == 0) count_list(a, all, copies);
    }
    if (!info[kAct]) return;
    const int* row = a.table + info[kRow] * a.M;
    const int* fresh = a.fresh + i * a.M;
    if (info[kGone]) {
        if (a.upto) upto = a.upto[2 * i];
        else before(a, kGone, i, lane, upto, all);
        int64_t at = (int64_t)list_len(a) + upto;
        for (int e0 = info[kFrom]; e0 < info[kHeld]; e0 += 64) {
            const int e = e0 + lane, p = e < info[kHeld] ? row[e] : -1;
            const bool gone = page_of(a, p) && gives_up(a, p, i, e);
            const uint64_t m = __ballot(gone);
            const int64_t to = at + __popcll(m & (((uint64_t)1 << lane) - 1));
            if (gone && to < a.N) a.free_pages[to] = p;
            at += __popcll(m);
        }
    }
    const int end = held_of(a, info[kLen]);
    for (int e = info[kFrom] + lane; e < info[kHeld] || e < end; e += 64) {
        const int old = e < info[kHeld] ? row[e] : -1, p = e < end ? fresh[e] : -1;
        if (page_of(a, old)) a.next[old] = next_shares(a, old);
        if (p >= 0) a.next[p] = next_shares(a, p);
    }
}

__device__ inline void fork_take(const ForkArgs& a, int i, int lane) {
    const int* info = a.info + 8 * i;
    if (i == 0 && lane == 0) *a.free_count = a.have[0] - a.have[1];
    int from = -1, to = -1, tokens = 0;
    if (info[kAct]) {
        const int r = info[kRow], len = info[kLen], whole = len / a.P;
        int* row = a.table + r * a.M;
        const int* fresh = a.fresh + i * a.M;
        int end = info[kEnd];
        if (info[kCopy]) {
            int upto, all;
            if (a.upto) upto = a.upto[2 * i + 1];
            else before(a, kCopy, i, lane, upto, all);
            if (upto < a.have[1]) {
                end = to = a.free_pages[a.have[0] - a.have[1] + upto];
                from = fresh[whole];
                tokens = len % a.P;
            }
        }
        const int held = info[kHeld], n = held > whole + 1 ? held : whole + 1, mine = held_of(a, len);
        for (int e = info[kFrom] + lane; e < n && e < a.M; e += 64) {
            const int old = e < held ? row[e] : -1, p = e < mine ? fresh[e] : -1;
            if (page_of(a, old)) a.shares[old] = a.next[old];
            if (p >= 0) a.shares[p] = a.next[p];
            row[e] = e < whole ? p : e == whole ? end : -1;
        }
        if (lane == 0) {
            const int n = end >= 0 ? len : whole * a.P;
            a.lens[r] = n;
            if (a.seq) a.seq[r] = n;
        }
    }
    if (lane < 3) a.copies[3 * i + lane] = lane == 0 ? from : lane == 1 ? to : tokens;
}

constexpr int kForkThreads = 1024, kStepThreads = 256;

__global__ __launch_bounds__(kForkThreads) void k_fork_one(ForkArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int W = kForkThreads / 64;
    for (int i = wave; i < a.n; i += W) fork_read(a, i, lane);
    __syncthreads();
    for (int i = wave; i < a.n; i += W) fork_count(a, i, lane);
    __syncthreads();
    for (int i = wave; i < a.n; i += W) fork_sum(a, i, lane);
    __syncthreads();
    for (int i = wave; i < a.n; i += W) fork_give(a, i, lane);
    __syncthreads();
    for (int i = wave; i < a.n; i += W) fork_take(a, i, lane);
}

template <int STEP>
__global__ __launch_bounds__(kStepThreads) void k_fork_step(ForkArgs a) {
    const int lane = threadIdx.x & 63;
    const int i = __builtin_amdgcn_readfirstlane(blockIdx.x * (kStepThreads / 64) + (threadIdx.x >> 6));
    if (i >= a.n) return;
    if constexpr (STEP == 0) fork_read(a, i, lane);
    if constexpr (STEP == 1) fork_count(a, i, lane);
    if constexpr (STEP == 2) fork_sum(a, i, lane);
    if constexpr (STEP == 3) fork_give(a, i, lane);
    if constexpr (STEP == 4) fork_take(a, i, lane);
}

// Threads: pairs.  The rows' names, cleared and then taken.
template <bool CLEAR>
__global__ __launch_bounds__(kStepThreads) void k_fork_name(ForkArgs a) {
    const int i = blockIdx.x * kStepThreads + threadIdx.x, r = i < a.n ? a.rows[i] : -1;
    if (r < 0 || r >= a.R) return;
    int* named = a.named + 2 * (int64_t)r;
    if constexpr (CLEAR) {
        named[0] = named[1] = kNone;
    } else {
        atomicMin(&named[0], i);
        atomicMin(&named[1], a.keep[i]);
    }
}

// One workgroup, neighbouring pairs a thread.  Copies in the upper half of a sum,
// pages in the lower: no page is given up twice, so neither passes 2^31.
__global__ __launch_bounds__(kForkThreads) void k_fork_upto(ForkArgs a) {
    constexpr int W = kForkThreads / 64;
    __shared__ uint64_t part[W];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (a.n + kForkThreads - 1) / kForkThreads, i0 = tid * per;
    auto of = [&](int i) { return (uint64_t)(uint32_t)a.info[8 * i + kCopy] << 32 | (uint32_t)a.info[8 * i + kGone]; };
    uint64_t mine = 0;
    for (int i = i0; i < i0 + per && i < a.n; ++i) mine += of(i);
    uint64_t x = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint64_t y = __shfl_up((unsigned long long)x, o);
        if (lane >= o) x += y;
    }
    if (lane == 63) part[wave] = x;
    __syncthreads();
    for (int w = 0; w < wave; ++w) x += part[w];
    if (tid == kForkThreads - 1) count_list(a, (int)(uint32_t)x, (int)(x >> 32));
    x -= mine;
    for (int i = i0; i < i0 + per && i < a.n; ++i) {
        a.upto[2 * i] = (int)(uint32_t)x;
        a.upto[2 * i + 1] = (int)(x >> 32);
        x += of(i);
    }
}

template <int STEP>
hipError_t fork_steps(const ForkArgs& a, hipStream_t s) {
    constexpr int W = kStepThreads / 64;
    const dim3 pairs((a.n + kStepThreads - 1) / kStepThreads);
    if (STEP == 0 && a.named) {
        k_fork_name<true><<<pairs, dim3(kStepThreads), 0, s>>>(a);
        k_fork_name<false><<<pairs, dim3(kStepThreads), 0, s>>>(a);
    }
    if (STEP == 3 && a.upto) k_fork_upto<<<dim3(1), dim3(kForkThreads), 0, s>>>(a);
    k_fork_step<STEP><<<dim3((a.n + W - 1) / W), dim3(kStepThreads), 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if constexpr (STEP < 4) return e == hipSuccess ? fork_steps<STEP + 1>(a, s) : e;
    return e;
}

// ---- compact ---------------------------------------------------------------------------
//
// Places are ranks: the k-th page to move goes to the k-th free one, and both are
// counted in a bitmap of the free pages, so that any thread finds any page's new
// number by itself.  4096 pages, 64 rows: 4.6 + 4.4 us, launches and dependent
// reads.

constexpr int kMarkThreads = 1024;

__device__ inline int list_len(const CompactArgs& a) {
    const int n = *a.free_count;
    return n < 0 ? 0 : n > a.N ? (int)a.N : n;
}

// One workgroup: a bit for every free page, and how many lie before each word.
__global__ __launch_bounds__(kMarkThreads) void k_compact_mark(CompactArgs a) {
    extern __shared__ uint32_t bits[];
    __shared__ int part[kMarkThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int words = (int)((a.N + 31) / 32), n = list_len(a);
    for (int i = tid; i < words; i += kMarkThreads) bits[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kMarkThreads) {
        const int p = a.free_pages[i];
        if (p >= 0 && p < a.N) atomicOr(&bits[p >> 5], 1u << (p & 31));
    }
    __syncthreads();
    const int per = (words + kMarkThreads - 1) / kMarkThreads, w0 = tid * per;
    int mine = 0;
    for (int i = w0; i < w0 + per && i < words; ++i) mine += __popc(bits[i]);
    int x = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(x, o);
        if (lane >= o) x += y;
    }
    if (lane == 63) part[wave] = x;
    __syncthreads();
    for (int w = 0; w < wave; ++w) x += part[w];
    int at = x - mine;
    for (int i = w0; i < w0 + per && i < words; ++i) {
        a.bits[i] = bits[i];
        a.before[i] = at;
        at += __popc(bits[i]);
    }
    if (tid == kMarkThreads - 1) a.before[words] = x;
}

// Free pages below page p.
__device__ inline int free_below(const CompactArgs& a, int p) {
    return a.before[p >> 5] + __popc(a.bits[p >> 5] & ((1u << (p & 31)) - 1));
}
__device__ inline bool is_free(const CompactArgs& a, int p) { return a.bits[p >> 5] >> (p & 31) & 1; }

// The k-th free page.
__device__ inline int free_at(const CompactArgs& a, int k, int words) {
    int lo = 0, hi = words;  // before[lo] <= k < before[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.before[mid] <= k) lo = mid;
        else hi = mid;
    }
    uint32_t b = a.bits[lo];
    for (k -= a.before[lo]; k > 0; --k) b &= b - 1;
    return lo * 32 + __builtin_ctz(b);
}

// Rank of a page in use among those from `used` on.
__device__ inline int mover_rank(const CompactArgs& a, int p, int used) {
    // pages in use below p, less those below `used`
    return (p - free_below(a, p)) - (used - (used < a.N ? free_below(a, used) : a.before[(a.N + 31) / 32]));
}

// Threads: entries of the table, then pages, then moves.
__global__ __launch_bounds__(256) void k_compact_apply(CompactArgs a) {
    const int words = (int)((a.N + 31) / 32);
    const int left = a.before[words], used = (int)a.N - left;
    const int64_t entries = a.R * a.M, step = (int64_t)gridDim.x * 256;
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < entries + a.N + a.n_moves; i += step) {
        if (i < entries) {
            const int64_t r = i / a.M;
            int p = a.table[i];
            const int len = a.lens[r];
            if (p >= used && p < a.N && len > 0 && (i - r * a.M) * a.P < len && !is_free(a, p))
                p = free_at(a, mover_rank(a, p, used), words);
            a.new_table[i] = p;
        } else if (i < entries + a.N) {
            const int p = (int)(i - entries);
            const bool free = is_free(a, p);
            if (p < left) a.new_free[p] = (int)a.N - 1 - p;
            if (p == 0) *a.free_left = left;
            if (p < used && !free) {
                a.new_shares[p] = a.shares[p];
            } else if (p >= used && !free) {
                // moved; nobody else reads or writes either place
                const int k = mover_rank(a, p, used), to = free_at(a, k, words);
                const int x = a.shares[p];
                a.new_shares[to] = x;
                a.new_shares[p] = 0;
                a.moves[3 * (int64_t)k] = p;
                a.moves[3 * (int64_t)k + 1] = to;
                a.moves[3 * (int64_t)k + 2] = a.P;
            } else if (p >= used) {
                a.new_shares[p] = 0;
            }
        } else {
            const int64_t k = i - entries - a.N;
            const int holes = used < a.N ? free_below(a, used) : left;
            if (k >= holes) {
                a.moves[3 * k] = a.moves[3 * k + 1] = -1;
                a.moves[3 * k + 2] = 0;
            }
        }
    }
}

// ---- copy --------------------------------------------------------------------------------

constexpr int kCopyThreads = 256, kCopyUnits = 1024;

// Bound by memory: 1024 pages of 66 KB 32 us, 4.3 TB/s read and written (a large
// copy: 4.7).
//
// Grid (entries, 16-byte units of codes in pieces of 1024).
__global__ __launch_bounds__(kCopyThreads) void k_kv4_copy(CopyArgs a) {
    const int32_t* c = a.copies + (int64_t)blockIdx.x * 3;
    const int src = c[0], dst = c[1];
    int tokens = c[2];
    if (src < 0 || src >= a.pages || dst < 0 || dst >= a.pages || tokens <= 0) return;
    tokens = tokens < a.P ? tokens : a.P;
    const int blocks = (tokens + kKvBlock - 1) / kKvBlock, all = a.P / kKvBlock;
    const int slabs = 2 * a.H;                      // k and v of each head
    const uint32_t per = (uint32_t)blocks * a.D;    // 16-byte units of codes of a slab
    const int64_t units = (int64_t)slabs * per;
    typedef uint32_t uintx4 __attribute__((ext_vector_type(4)));
    const uintx4* from = reinterpret_cast<const uintx4*>(a.codes) + (int64_t)src * slabs * all * a.D;
    uintx4* to = reinterpret_cast<uintx4*>(a.codes) + (int64_t)dst * slabs * all * a.D;
    const int64_t u0 = (int64_t)blockIdx.y * kCopyUnits;
    uintx4 x[kCopyUnits / kCopyThreads];
    int64_t at[kCopyUnits / kCopyThreads];
#pragma unroll
    for (int i = 0; i < kCopyUnits / kCopyThreads; ++i) {
        const int64_t u = u0 + i * kCopyThreads + threadIdx.x;
        const uint32_t slab = (uint32_t)u / per;
        at[i] = u < units ? (int64_t)slab * all * a.D + ((uint32_t)u - slab * per) : -1;
        if (at[i] >= 0) x[i] = from[at[i]];
    }
#pragma unroll
    for (int i = 0; i < kCopyUnits / kCopyThreads; ++i)
        if (at[i] >= 0) to[at[i]] = x[i];
    if (blockIdx.y) return;
    const uintx4* sf = reinterpret_cast<const uintx4*>(a.scales) + (int64_t)src * slabs * (a.P / 8);
    uintx4* st = reinterpret_cast<uintx4*>(a.scales) + (int64_t)dst * slabs * (a.P / 8);
    const int each = blocks * (kKvBlock / 8);
    for (int i = threadIdx.x; i < slabs * each; i += kCopyThreads) {
        const int slab = i / each, k = slab * (a.P / 8) + (i - slab * each);
        st[k] = sf[k];
    }
}

}  // namespace

hipError_t launch_kv_fork(const ForkArgs& a, hipStream_t s) {
    // One workgroup has 16 waves: rows of 64 entries, four a wave, take its steps
    // less time than four launches more.
    if (a.n <= 64 && a.n * a.M <= 64 * 256) {
        k_fork_one<<<dim3(1), dim3(kForkThreads), 0, s>>>(a);
        return hipGetLastError();
    }
    return fork_steps<0>(a, s);
}

hipError_t launch_kv_compact(const CompactArgs& a, hipStream_t s) {
    static LdsAttr rec;
    const int lds = (int)((a.N + 31) / 32 * 4);
    hipError_t e = ensure_lds(rec, reinterpret_cast<const void*>(k_compact_mark), 131072);
    if (e != hipSuccess) return e;
    k_compact_mark<<<dim3(1), dim3(kMarkThreads), lds, s>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t n = (a.R * a.M + a.N + a.n_moves + 255) / 256;
    k_compact_apply<<<dim3((unsigned)(n < 4096 ? n : 4096)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_kv4_copy(const CopyArgs& a, hipStream_t s) {
    const int64_t units = (int64_t)2 * a.H * (a.P / kKvBlock) * a.D;
    k_kv4_copy<<<dim3((unsigned)a.n, (unsigned)((units + kCopyUnits - 1) / kCopyUnits)),
                 dim3(kCopyThreads), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace fk
