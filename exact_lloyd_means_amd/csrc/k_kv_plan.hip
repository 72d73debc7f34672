// k_kv_plan.hip -- block tables and slot maps of a serving step (fk_kv_plan).
//
// With seq = ctx + new, held = ceil(ctx / P) and need = max(0, min(ceil(seq /
// P), M) - held), the two exclusive prefix sums over requests, of new and of
// need, decide everything: token i of the step belongs to the request whose
// range of the first holds i, and its page is either in the table already or
// number off_b + (page - held_b) of the pages taken from the free list.
//
// Nothing here is heavy; a call is bound by latency (dependent loads and
// launches).  One workgroup does the scans.  Where the tokens are few it also
// fills tables and slots from LDS in the same launch; else a second launch
// fills them from many workgroups, each token's request found by a search in
// the prefix sums.  64 requests: 4.7 us; 3000 requests and 2^20 slots, 8.5 MB:
// 6.4 and 9.4 us.
#include "kv4_internal.h"

namespace fk {
namespace {

constexpr int64_t kSat = 2147483647;

// One launch up to this many requests (12 bytes of LDS each) and tokens; a
// quarter of a workgroup's threads up to the smaller numbers (64 requests and
// tokens: 7.6 -> 4.4 us).
constexpr int kOneB = 4096, kSmallB = 1024;
constexpr int64_t kOneTokens = 16384, kSmallTokens = 2048;

__device__ inline int32_t sat(int64_t x) { return (int32_t)(x > kSat ? kSat : x); }
// Sums that stop at 2^32 - 1: those below 2^31 are right, others are large.
__device__ inline uint32_t add(uint32_t x, uint32_t y) { return __builtin_elementwise_add_sat(x, y); }
__device__ inline int32_t low(uint32_t x) { return (int32_t)(x > (uint32_t)kSat ? (uint32_t)kSat : x); }

__device__ inline uint32_t wave_scan(uint32_t x, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const uint32_t y = __shfl_up(x, o);
        if (lane >= o) x = add(x, y);
    }
    return x;
}

// New token t of request b: its position, and where its page is to be read
// (null: there is none).  In two parts, so that several tokens' reads overlap.
struct Spot {
    const int32_t* from;
    uint32_t pg, in, pos;
    bool fresh;  // the page is one of the list's
};
__device__ inline Spot locate(const PlanArgs& a, int64_t t, int64_t b, int32_t cu, int32_t ctx,
                              int32_t off, int32_t n) {
    const uint32_t P = (uint32_t)a.page_size;
    const int64_t pos64 = (int64_t)ctx + (t - cu);
    Spot s;
    s.pos = (uint32_t)(pos64 > kSat ? kSat : pos64);
    s.pg = s.pos / P;
    s.in = s.pos - s.pg * P;
    const uint32_t held = ((uint32_t)ctx + P - 1) / P;
    s.fresh = s.pg >= held && (int64_t)s.pg < a.max_pages;
    const int64_t i = (int64_t)n - 1 - off - (int64_t)(s.pg - held);
    s.from = s.fresh ? (i >= 0 ? a.free_pages + i : nullptr)
                     : s.pg < held && (int64_t)s.pg < a.max_pages ? a.table + b * a.max_pages + s.pg
                                                                  : nullptr;
    return s;
}
// Slot (t < slot_cap) and, for the first token of a fresh page, table entry.
__device__ inline void place(const PlanArgs& a, int64_t t, int64_t b, const Spot& s, int32_t page) {
    if (s.fresh && s.in == 0) a.table[b * a.max_pages + s.pg] = page;
    const int64_t slot = (int64_t)page * a.page_size + s.in;
    a.slots[t] = page >= 0 && slot <= kSat ? (int32_t)slot : -1;
    if (a.pos) a.pos[t] = (int32_t)s.pos;
}

// Table entries of needed pages first, first + stride, ...: where there are
// more tokens than slots, so that a step's work follows its slots and pages and
// not the tokens without a slot.  off: a request's first needed page.
template <typename Off, typename Ctx>
__device__ inline void place_pages(const PlanArgs& a, int64_t first, int64_t stride, int64_t wanted,
                                   int32_t n, Off off, Ctx ctx) {
    const uint32_t P = (uint32_t)a.page_size;
    for (int64_t i = first; i < wanted; i += stride) {
        int64_t lo = 0, hi = a.B;  // off(lo) <= i < off(hi): the last of those that need none is passed
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) >> 1;
            if (off(mid) <= i) lo = mid;
            else hi = mid;
        }
        const uint32_t held = ((uint32_t)ctx(lo) + P - 1) / P;
        a.table[lo * a.max_pages + held + (i - off(lo))] = i < n ? a.free_pages[n - 1 - i] : -1;
    }
}

__device__ inline void no_token(const PlanArgs& a, int64_t t) {
    a.slots[t] = -1;
    if (a.pos) a.pos[t] = -1;
}

// Scans over all requests by one workgroup of N threads, four consecutive
// requests a thread and round.  FILL: the fills too (B <= 4 N).
template <int N, bool FILL>
__global__ __launch_bounds__(N) void k_plan_scan(PlanArgs a) {
    constexpr int kWaves = N / kWave, kB = FILL ? 4 * N : 1;
    __shared__ uint32_t s_tok[kWaves], s_page[kWaves], s_lost[kWaves];
    __shared__ int32_t s_cu[kB + 1], s_off[kB], s_ctx[kB];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t P = (uint32_t)a.page_size;
    const int64_t M = a.max_pages;
    const int32_t n0 = *a.free_count;
    const uint32_t n = n0 < 0 ? 0 : (uint32_t)(n0 > a.free_cap ? a.free_cap : n0);
    uint32_t tok0 = 0, page0 = 0, lost = 0;
    for (int64_t base = 0; base < a.B; base += 4 * N) {
        uint32_t ctx[4], fresh[4], need[4], held[4], tok = 0, pages = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t b = base + 4 * tid + e;
            const bool on = b < a.B;
            const int32_t c = on ? a.ctx[b] : 0, f = on ? a.fresh[b] : 0;
            ctx[e] = c < 0 ? 0 : c;
            fresh[e] = f < 0 ? 0 : f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            held[e] = (ctx[e] + P - 1) / P;
            const uint32_t all = ((uint32_t)low(ctx[e] + fresh[e]) + P - 1) / P;
            const uint32_t want = all < M ? all : (uint32_t)M;
            need[e] = want > held[e] ? want - held[e] : 0;
            tok = add(tok, fresh[e]);
            pages = add(pages, need[e]);
        }
        const uint32_t it = wave_scan(tok, lane), ip = wave_scan(pages, lane);
        if (lane == 63) {
            s_tok[wave] = it;
            s_page[wave] = ip;
        }
        // what lies before this thread: saturated sums cannot be subtracted
        uint32_t t = __shfl_up(it, 1), p = __shfl_up(ip, 1);
        if (lane == 0) t = p = 0;
        __syncthreads();
        t = add(t, tok0);
        p = add(p, page0);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const uint32_t x = s_tok[w], y = s_page[w];
            if (w < wave) {
                t = add(t, x);
                p = add(p, y);
            }
            tok0 = add(tok0, x);
            page0 = add(page0, y);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t b = base + 4 * tid + e;
            if (b < a.B) {
                a.cu[b] = low(t);
                a.seq[b] = low(ctx[e] + fresh[e]);
                if constexpr (FILL) {
                    s_cu[b] = low(t);
                    s_off[b] = low(p);
                    s_ctx[b] = (int32_t)ctx[e];
                } else {
                    a.ws[b] = low(p);
                }
                // pages of this request that the list still holds, and the
                // tokens past the last of them
                const uint32_t rest = n > p ? n - p : 0, got = rest < need[e] ? rest : need[e];
                const int64_t end = ((held[e] < M ? held[e] : M) + got) * (int64_t)P;
                const int64_t room = end > ctx[e] ? end : ctx[e];
                const int64_t miss = (int64_t)ctx[e] + fresh[e] - room;
                lost = add(lost, miss > 0 ? (uint32_t)miss : 0);
                if (a.kept) a.kept[b] = sat(miss > 0 ? room : (int64_t)ctx[e] + fresh[e]);
            }
            t = add(t, fresh[e]);
            p = add(p, need[e]);
        }
        if (base + 4 * N < a.B) __syncthreads();
    }
    const uint32_t total = tok0, wanted = page0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) lost = add(lost, __shfl_xor(lost, o));
    if (lane == 0) s_lost[wave] = lost;
    if constexpr (FILL)
        if (tid == 0) s_cu[a.B] = low(total);
    __syncthreads();
    if (tid == 0) {
        uint32_t all = 0;
        for (int w = 0; w < kWaves; ++w) all = add(all, s_lost[w]);
        const uint32_t taken = wanted < n ? wanted : n;
        a.cu[a.B] = low(total);
        a.free_left[0] = (int32_t)(n - taken);
        a.status[0] = low(total);
        a.status[1] = (int32_t)taken;
        a.status[2] = low(wanted - taken);
        a.status[3] = low(all);
        if constexpr (!FILL) a.ws[a.B] = (int32_t)n;
    }
    if constexpr (FILL) {
        const int64_t tot = low(total);
        for (int64_t t = tid; t < a.slot_cap; t += N) {
            if (t >= tot) {
                no_token(a, t);
                continue;
            }
            int lo = 0, hi = (int)a.B;  // s_cu[lo] <= t < s_cu[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_cu[mid] <= t) lo = mid;
                else hi = mid;
            }
            const Spot sp = locate(a, t, lo, s_cu[lo], s_ctx[lo], s_off[lo], (int32_t)n);
            place(a, t, lo, sp, sp.from ? *sp.from : -1);
        }
        if (tot > a.slot_cap)
            place_pages(a, tid, N, low(wanted), (int32_t)n, [&](int64_t b) { return s_off[b]; },
                        [&](int64_t b) { return s_ctx[b]; });
    }
}

// The largest b with cu[b] <= t for two t at once, by one wave: 64 probes a
// step, both loads of a step in flight together.
__device__ inline void wave_find(const int32_t* cu, int64_t B, int64_t t0, int64_t t1, int lane,
                                 int64_t& b0, int64_t& b1) {
    int64_t lo[2] = {0, 0}, len[2] = {B + 1, B + 1};
    const int64_t t[2] = {t0, t1};
    while (len[0] > 1 || len[1] > 1) {
        int64_t step[2];
        int32_t v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            step[i] = (len[i] + 63) / 64;
            const int64_t at = lane * step[i];
            v[i] = cu[lo[i] + (at < len[i] ? at : 0)];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t k = __popcll(__ballot(lane * step[i] < len[i] && v[i] <= t[i])) - 1;
            lo[i] += k * step[i];
            len[i] = len[i] - k * step[i] < step[i] ? len[i] - k * step[i] : step[i];
        }
    }
    b0 = lo[0];
    b1 = lo[1];
}

constexpr int kFillThreads = 256, kFillTokens = 1024, kFillB = 2048;

// 1024 tokens a workgroup and round; the prefix sums of their requests in LDS
// (more than kFillB of them only where most are idle).
__global__ __launch_bounds__(kFillThreads) void k_plan_fill(PlanArgs a) {
    __shared__ int32_t s_cu[kFillB];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t total = a.cu[a.B];
    const int32_t n = a.ws[a.B];
    for (int64_t t0 = (int64_t)blockIdx.x * kFillTokens; t0 < a.slot_cap;
         t0 += (int64_t)gridDim.x * kFillTokens) {
        int64_t b0 = 0, b1 = 0;
        if (t0 < total) {
            int64_t t1 = t0 + kFillTokens < total ? t0 + kFillTokens : total;
            t1 = t1 < a.slot_cap ? t1 : a.slot_cap;
            wave_find(a.cu, a.B, t0, t1 - 1, lane, b0, b1);
        }
        const bool staged = b1 - b0 < kFillB;
        if (b1 > b0 && staged) {
            __syncthreads();
            for (int64_t i = tid; i <= b1 - b0; i += kFillThreads) s_cu[i] = a.cu[b0 + i];
            __syncthreads();
        }
        constexpr int kEach = kFillTokens / kFillThreads;
        int64_t b[kEach];
        Spot sp[kEach];
        int32_t page[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int64_t t = t0 + tid + e * kFillThreads;
            sp[e].from = nullptr;
            if (t >= total || t >= a.slot_cap) continue;
            int64_t lo = b0, hi = b1 + 1;
            if (staged) {
                int l = 0, h = (int)(hi - lo);
                while (h - l > 1) {
                    const int mid = (l + h) >> 1;
                    if (s_cu[mid] <= t) l = mid;
                    else h = mid;
                }
                lo += l;
            } else {
                while (hi - lo > 1) {
                    const int64_t mid = (lo + hi) >> 1;
                    if (a.cu[mid] <= t) lo = mid;
                    else hi = mid;
                }
            }
            b[e] = lo;
        }
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int64_t t = t0 + tid + e * kFillThreads;
            if (t >= total || t >= a.slot_cap) continue;
            const int32_t c = a.ctx[b[e]];
            sp[e] = locate(a, t, b[e], a.cu[b[e]], c < 0 ? 0 : c, a.ws[b[e]], n);
        }
#pragma unroll
        for (int e = 0; e < kEach; ++e) page[e] = sp[e].from ? *sp[e].from : -1;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int64_t t = t0 + tid + e * kFillThreads;
            if (t >= a.slot_cap) continue;
            if (t < total) place(a, t, b[e], sp[e], page[e]);
            else no_token(a, t);
        }
    }
    if (total > a.slot_cap)  // pages wanted: taken and not there
        place_pages(a, (int64_t)blockIdx.x * kFillThreads + tid, (int64_t)gridDim.x * kFillThreads,
                    (int64_t)a.status[1] + a.status[2], n, [&](int64_t b) { return a.ws[b]; },
                    [&](int64_t b) { return a.ctx[b] < 0 ? 0 : a.ctx[b]; });
}

}  // namespace

hipError_t launch_kv_plan(const PlanArgs& a, hipStream_t s) {
    if (a.B <= kSmallB && a.slot_cap <= kSmallTokens) {
        k_plan_scan<256, true><<<dim3(1), dim3(256), 0, s>>>(a);
        return hipGetLastError();
    }
    if (a.B <= kOneB && a.slot_cap <= kOneTokens) {
        k_plan_scan<1024, true><<<dim3(1), dim3(1024), 0, s>>>(a);
        return hipGetLastError();
    }
    k_plan_scan<1024, false><<<dim3(1), dim3(1024), 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    int64_t wgs = (a.slot_cap + kFillTokens - 1) / kFillTokens;
    wgs = wgs < 64 ? 64 : wgs > 4096 ? 4096 : wgs;  // few slots: there may be pages all the same
    k_plan_fill<<<dim3((unsigned)wgs), dim3(kFillThreads), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace fk
