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
// the prefix sums.
#include "kv4_internal.h"

namespace fk {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kScanWaves = kScanThreads / kWave;
constexpr int64_t kSat = 2147483647;

// One launch up to this many requests (12 bytes of LDS each) and tokens.
constexpr int kSmallB = 4096;
constexpr int64_t kSmallTokens = 16384;

__device__ inline int32_t sat(int64_t x) { return (int32_t)(x > kSat ? kSat : x); }

__device__ inline int64_t wave_scan(int64_t x, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int64_t y = __shfl_up(x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// Slot and, for the first token of a fresh page, table entry of new token t
// of request b.
__device__ inline void place(const PlanArgs& a, int64_t t, int64_t b, int32_t cu, int32_t ctx,
                             int32_t off, int32_t n) {
    const uint32_t P = (uint32_t)a.page_size;
    const int64_t pos64 = (int64_t)ctx + (t - cu);
    const uint32_t pos = (uint32_t)(pos64 > kSat ? kSat : pos64);
    const uint32_t pg = pos / P, in = pos - pg * P;
    const uint32_t held = ((uint32_t)ctx + P - 1) / P;
    int32_t page = -1;
    if ((int64_t)pg < a.max_pages) {
        if (pg < held) {
            page = a.table[b * a.max_pages + pg];
        } else {
            const int64_t i = (int64_t)n - 1 - off - (int64_t)(pg - held);
            page = i >= 0 ? a.free_pages[i] : -1;
            if (in == 0) a.table[b * a.max_pages + pg] = page;
        }
    }
    if (t < a.slot_cap) {
        const int64_t slot = (int64_t)page * P + in;
        a.slots[t] = page >= 0 && slot <= kSat ? (int32_t)slot : -1;
        if (a.pos) a.pos[t] = (int32_t)pos;
    }
}

__device__ inline void no_token(const PlanArgs& a, int64_t t) {
    a.slots[t] = -1;
    if (a.pos) a.pos[t] = -1;
}

// Scans over all requests by one workgroup, four consecutive requests a
// thread and round.  FILL: the fills too (B <= kSmallB).
template <bool FILL>
__global__ __launch_bounds__(kScanThreads) void k_plan_scan(PlanArgs a) {
    __shared__ int64_t s_tok[kScanWaves], s_page[kScanWaves], s_lost[kScanWaves];
    __shared__ int32_t s_cu[FILL ? kSmallB + 1 : 1], s_off[FILL ? kSmallB : 1],
        s_ctx[FILL ? kSmallB : 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t P = a.page_size, M = a.max_pages;
    int32_t n0 = *a.free_count;
    const int64_t n = n0 < 0 ? 0 : n0 > a.free_cap ? a.free_cap : n0;
    int64_t tok0 = 0, page0 = 0, lost = 0;
    for (int64_t base = 0; base < a.B; base += 4 * kScanThreads) {
        int64_t ctx[4], fresh[4], need[4], tok = 0, pages = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t b = base + 4 * tid + e;
            const bool on = b < a.B;
            const int32_t c = on ? a.ctx[b] : 0, f = on ? a.fresh[b] : 0;
            ctx[e] = c < 0 ? 0 : c;
            fresh[e] = f < 0 ? 0 : f;
            const int64_t held = (int64_t)(((uint32_t)ctx[e] + (uint32_t)P - 1) / (uint32_t)P);
            int64_t want = ((uint32_t)sat(ctx[e] + fresh[e]) + (uint32_t)P - 1) / (uint32_t)P;
            want = want > M ? M : want;
            need[e] = want > held ? want - held : 0;
            tok += fresh[e];
            pages += need[e];
        }
        const int64_t it = wave_scan(tok, lane), ip = wave_scan(pages, lane);
        if (lane == 63) {
            s_tok[wave] = it;
            s_page[wave] = ip;
        }
        __syncthreads();
        int64_t bt = tok0, bp = page0;
#pragma unroll
        for (int w = 0; w < kScanWaves; ++w) {
            const int64_t x = s_tok[w], y = s_page[w];
            if (w < wave) {
                bt += x;
                bp += y;
            }
            tok0 += x;
            page0 += y;
        }
        int64_t t = bt + it - tok, p = bp + ip - pages;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t b = base + 4 * tid + e;
            if (b < a.B) {
                a.cu[b] = sat(t);
                a.seq[b] = sat(ctx[e] + fresh[e]);
                if constexpr (FILL) {
                    s_cu[b] = sat(t);
                    s_off[b] = sat(p);
                    s_ctx[b] = (int32_t)ctx[e];
                } else {
                    a.ws[b] = sat(p);
                }
                // pages of this request that the list still holds, and the
                // tokens past the last of them
                int64_t got = n - p;
                got = got < 0 ? 0 : got > need[e] ? need[e] : got;
                int64_t held = (ctx[e] + P - 1) / P;
                held = held > M ? M : held;
                const int64_t end = (held + got) * P;
                const int64_t miss = ctx[e] + fresh[e] - (end > ctx[e] ? end : ctx[e]);
                lost += miss > 0 ? miss : 0;
            }
            t += fresh[e];
            p += need[e];
        }
        __syncthreads();
    }
    const int64_t total = tok0, wanted = page0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) lost += __shfl_xor(lost, o);
    if (lane == 0) s_lost[wave] = lost;
    if constexpr (FILL)
        if (tid == 0) s_cu[a.B] = sat(total);
    __syncthreads();
    if (tid == 0) {
        int64_t all = 0;
        for (int w = 0; w < kScanWaves; ++w) all += s_lost[w];
        const int64_t taken = wanted < n ? wanted : n;
        a.cu[a.B] = sat(total);
        a.free_left[0] = (int32_t)(n - taken);
        a.status[0] = sat(total);
        a.status[1] = (int32_t)taken;
        a.status[2] = sat(wanted - taken);
        a.status[3] = sat(all);
        if constexpr (!FILL) a.ws[a.B] = (int32_t)n;
    }
    if constexpr (FILL) {
        const int64_t tot = sat(total), last = tot > a.slot_cap ? tot : a.slot_cap;
        for (int64_t t = tid; t < last; t += kScanThreads) {
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
            place(a, t, lo, s_cu[lo], s_ctx[lo], s_off[lo], (int32_t)n);
        }
    }
}

// The largest b with cu[b] <= t, by one wave: 64 probes a step.
__device__ inline int64_t wave_find(const int32_t* cu, int64_t B, int64_t t, int lane) {
    int64_t lo = 0, len = B + 1;
    while (len > 1) {
        const int64_t step = (len + 63) / 64, at = lane * step;
        const uint64_t m = __ballot(at < len && cu[lo + (at < len ? at : 0)] <= t);
        const int64_t k = __popcll(m) - 1;
        lo += k * step;
        len = len - k * step < step ? len - k * step : step;
    }
    return lo;
}

constexpr int kFillThreads = 256, kFillTokens = 1024;

__global__ __launch_bounds__(kFillThreads) void k_plan_fill(PlanArgs a) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t total = a.cu[a.B];
    const int32_t n = a.ws[a.B];
    const int64_t last = total > a.slot_cap ? total : a.slot_cap;
    for (int64_t t0 = (int64_t)blockIdx.x * kFillTokens; t0 < last;
         t0 += (int64_t)gridDim.x * kFillTokens) {
        int64_t b0 = 0, b1 = 0;
        if (t0 < total) {
            const int64_t t1 = t0 + kFillTokens < total ? t0 + kFillTokens : total;
            b0 = wave_find(a.cu, a.B, t0, lane);
            b1 = wave_find(a.cu, a.B, t1 - 1, lane);
        }
        for (int64_t t = t0 + tid; t < t0 + kFillTokens && t < last; t += kFillThreads) {
            if (t >= total) {
                no_token(a, t);
                continue;
            }
            int64_t lo = b0, hi = b1 + 1;
            while (hi - lo > 1) {
                const int64_t mid = (lo + hi) >> 1;
                if (a.cu[mid] <= t) lo = mid;
                else hi = mid;
            }
            const int32_t c = a.ctx[lo];
            place(a, t, lo, a.cu[lo], c < 0 ? 0 : c, a.ws[lo], n);
        }
    }
}

}  // namespace

hipError_t launch_kv_plan(const PlanArgs& a, hipStream_t s) {
    if (a.B <= kSmallB && a.slot_cap <= kSmallTokens) {
        k_plan_scan<true><<<dim3(1), dim3(kScanThreads), 0, s>>>(a);
        return hipGetLastError();
    }
    k_plan_scan<false><<<dim3(1), dim3(kScanThreads), 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    int64_t wgs = (a.slot_cap + kFillTokens - 1) / kFillTokens;
    wgs = wgs < 1 ? 1 : wgs > 4096 ? 4096 : wgs;
    k_plan_fill<<<dim3((unsigned)wgs), dim3(kFillThreads), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace fk
