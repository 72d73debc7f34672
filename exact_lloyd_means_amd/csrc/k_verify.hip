// k_verify.hip -- which drafted tokens the target keeps (fk_verify).
//
// Weights count in multiples of 2^-42, as 64-bit integers: with V <= 2^20 and
// weights up to 1 a sum stays below 2^62 and is exact, so the rows can be cut
// and summed in any order and the token found is the same.
//
// Two launches: k_verify_sums cuts the one row that a request samples from into
// pieces, one a wave, and sums each (for greedy decoding k_verify_best the
// largest values of all rows), k_verify_pick finds the piece that holds the
// point and searches that piece alone.  Bound by memory for many requests: one
// row of the target and one of the draft a request are read once (64 requests of
// 128000 tokens in fp32: 13.8 us, 4.7 TB/s), then by the chain sums, piece, token
// (5.7 us; 8.9 with pieces of a workgroup, whose search reads four times as
// much); for few by two launches of that chain (4.1 + 4.0 us).  Greedy (32
// requests, 98 rows of 150001 in bf16: 9.0 + 3.9 us traced, 11.2 a call) by
// k_verify_best's 64-bit keys and four loads a thread that follow each other;
// memory alone would take 5.2.
#include "serve_internal.h"

namespace fk {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

template <int DT>
struct Elem {
    typedef uint16_t type;
    static constexpr int kVec = 8;
    static __device__ inline float get(uint16_t x) { return kv_f32<DT>(x); }
};
template <>
struct Elem<FK_F32> {
    typedef float type;
    static constexpr int kVec = 4;
    static __device__ inline float get(float x) { return x; }
};
// Rows start anywhere: 16 bytes at the alignment of an element.
template <int DT>
struct __attribute__((packed, aligned(sizeof(typename Elem<DT>::type)))) Piece {
    typename Elem<DT>::type e[Elem<DT>::kVec];
};

__device__ inline uint64_t weight(float x) {
    x = x > 0.f ? x : 0.f;  // NaN too
    x = x < 1.f ? x : 1.f;
    return (uint64_t)(x * 4398046511104.f);  // 2^42: exact
}

struct Rows {
    int first, n;
};
__device__ inline Rows rows_of(const VerifyArgs& a, int b) {
    const int T = (int)a.T;
    int c0 = a.cu[b], c1 = a.cu[b + 1];
    c0 = c0 < 0 ? 0 : c0 > T ? T : c0;
    c1 = c1 < c0 ? c0 : c1 > T ? T : c1;
    return {c0, c1 - c0};
}

// Drafts kept of a request, up to its first row whose draft is refused, or the
// last; times two, and one more unless that draft is no token.  `least` in LDS;
// all threads call it.
template <int DT>
__device__ inline int kept(const VerifyArgs& a, const Rows& r, int* least, int threads) {
    typedef typename Elem<DT>::type E;
    if (threadIdx.x == 0) *least = 2 * (r.n - 1) + 1;
    __syncthreads();
    for (int i = threadIdx.x; i < r.n - 1; i += threads) {
        if (i >= *(volatile int*)least / 2) break;
        const int64_t row = r.first + i;
        const int d = a.tokens[row + 1];
        const bool token = d >= 0 && d < a.V;
        bool good = token;
        if (good) {
            const float p = Elem<DT>::get(static_cast<const E*>(a.p)[row * a.p_row + d]);
            const float q = a.q ? Elem<DT>::get(static_cast<const E*>(a.q)[row * a.q_row + d]) : 1.f;
            good = (double)a.u[row] * (double)q < (double)p;  // 48 bits: exact
        }
        if (!good) atomicMin(least, 2 * i + token);
    }
    __syncthreads();
    return *least;
}

// What the token of a row is drawn from.
template <int DT>
struct Source {
    const typename Elem<DT>::type *p, *q;  // q null: nothing is taken away
    int without;                           // or this token is, alone; -1: none
};
template <int DT>
__device__ inline Source<DT> source(const VerifyArgs& a, const Rows& r, int kept) {
    typedef typename Elem<DT>::type E;
    const int64_t row = r.first + kept / 2;
    Source<DT> s{static_cast<const E*>(a.p) + row * a.p_row, nullptr, -1};
    // a draft that is no token was drawn from nothing: there is nothing to take away
    if (kept / 2 < r.n - 1 && kept % 2) {
        if (a.q) s.q = static_cast<const E*>(a.q) + row * a.q_row;
        else s.without = a.tokens[row + 1];
    }
    return s;
}

// Weights of what is left and of p for elements i .. i + kVec - 1, none from hi on.
template <int DT>
__device__ inline void weights(const Source<DT>& s, int64_t i, int64_t hi,
                               uint64_t (&left)[Elem<DT>::kVec], uint64_t (&plain)[Elem<DT>::kVec]) {
    typedef typename Elem<DT>::type E;
    constexpr int N = Elem<DT>::kVec;
    Piece<DT> p, q;
    if (i + N <= hi) {
        p = *reinterpret_cast<const Piece<DT>*>(s.p + i);
        if (s.q) q = *reinterpret_cast<const Piece<DT>*>(s.q + i);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            p.e[e] = i + e < hi ? s.p[i + e] : E(0);
            if (s.q) q.e[e] = i + e < hi ? s.q[i + e] : E(0);
        }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float x = Elem<DT>::get(p.e[e]);
        left[e] = plain[e] = weight(x);
        if (s.q) left[e] = weight(x - Elem<DT>::get(q.e[e]));
        else if (i + e == s.without) left[e] = 0;
    }
}

__device__ inline uint64_t wave_sum(uint64_t x) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor((unsigned long long)x, o);
    return x;
}

// Grid (four pieces, requests in two dimensions).
template <int DT>
__global__ __launch_bounds__(kThreads) void k_verify_sums(VerifyArgs a) {
    __shared__ int least;
    const int b = blockIdx.y + blockIdx.z * gridDim.y, tid = threadIdx.x, lane = tid & 63;
    if (b >= a.B) return;
    const Rows r = rows_of(a, b);
    if (r.n <= 0) return;
    const int j = kept<DT>(a, r, &least, kThreads);
    const Source<DT> s = source<DT>(a, r, j);
    const int piece = blockIdx.x * kWaves + (tid >> 6);
    const int64_t lo = (int64_t)piece * a.len, hi = lo + a.len < a.V ? lo + a.len : a.V;
    uint64_t left = 0, plain = 0;
    constexpr int N = Elem<DT>::kVec;
    for (int64_t i = lo + lane * N; i < hi; i += 64 * N) {
        uint64_t x[N], y[N];
        weights<DT>(s, i, hi, x, y);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            left += x[e];
            plain += y[e];
        }
    }
    left = wave_sum(left);
    plain = wave_sum(plain);
    if (lane == 0 && piece < a.pieces) {
        uint64_t* to = a.sums + ((int64_t)b * a.pieces + piece) * 2;
        to[0] = left;
        to[1] = plain;
        if (piece == 0) a.kept[b] = j;
    }
}

// Drafts, token and length of a request.
__device__ inline void tell(const VerifyArgs& a, int b, const Rows& r, int accepted, int token,
                            int threads) {
    for (int i = threadIdx.x; i < r.n; i += threads)
        a.emitted[r.first + i] = i < accepted ? a.tokens[r.first + i + 1] : i == accepted ? token : -1;
    if (threadIdx.x == 0) {
        a.accepted[b] = accepted;
        if (a.keep) a.keep[b] = a.seq[b] - (r.n > 0 ? r.n - 1 - accepted : 0);
    }
}

// Inclusive sums over the threads of a workgroup.
__device__ inline uint64_t group_scan(uint64_t x, uint64_t* scratch, uint64_t& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint64_t y = __shfl_up((unsigned long long)x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // scratch may still be read
    if (lane == 63) scratch[wave] = x;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const uint64_t y = scratch[w];
        if (w < wave) x += y;
        total += y;
    }
    return x;
}

// Grid: requests.  The piece whose inclusive sum first exceeds the point, then
// the element in it.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_verify_pick(VerifyArgs a) {
    __shared__ int found;
    __shared__ uint64_t scratch[kWaves], before;
    const int b = blockIdx.x, tid = threadIdx.x;
    const Rows r = rows_of(a, b);
    if (r.n <= 0) {
        tell(a, b, r, 0, -1, kThreads);
        return;
    }
    const int j = a.kept[b];
    const Source<DT> s = source<DT>(a, r, j);
    // a thread's pieces lie side by side
    const int per = (a.pieces + kThreads - 1) / kThreads, p0 = tid * per;
    const uint64_t* sums = a.sums + (int64_t)b * a.pieces * 2;
    uint64_t x = 0, y = 0, total;
    for (int i = p0; i < p0 + per && i < a.pieces; ++i) {
        x += sums[2 * i];
        y += sums[2 * i + 1];
    }
    uint64_t upto = group_scan(x, scratch, total);
    const bool plain = total == 0;  // nothing is left: p itself
    if (plain) {
        x = y;
        upto = group_scan(x, scratch, total);
    }
    int token = -1;
    if (total > 0) {
        const float u = a.pick[b];
        uint32_t k = u > 0.f ? (u < 1.f ? (uint32_t)(u * 2147483648.f) : 0x7fffffffu) : 0u;
        k = k > 0x7fffffffu ? 0x7fffffffu : k;
        // floor(k total / 2^31)
        const uint64_t point = 2 * (total >> 32) * k + ((total & 0xffffffffu) * k >> 31);
        if (upto > point && upto - x <= point) {
            uint64_t at = upto - x;
            int i = p0;
            for (;; ++i) {
                const uint64_t z = sums[2 * i + (plain ? 1 : 0)];
                if (at + z > point) break;
                at += z;
            }
            found = i;
            before = at;
        }
        __syncthreads();
        const int64_t lo = (int64_t)found * a.len, hi = lo + a.len < a.V ? lo + a.len : a.V;
        uint64_t base = before;
        __syncthreads();
        constexpr int N = Elem<DT>::kVec;
        for (int64_t at = lo; at < hi; at += kThreads * N) {
            uint64_t w[N], p[N], mine = 0, sum;
            const int64_t i = at + tid * N;
            weights<DT>(s, i, hi, w, p);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                w[e] = plain ? p[e] : w[e];
                mine += w[e];
            }
            const uint64_t up = base + group_scan(mine, scratch, sum);
            if (up > point && up - mine <= point) {
                uint64_t z = up - mine;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    if (z <= point && z + w[e] > point) found = (int)(i + e);
                    z += w[e];
                }
            }
            base += sum;
            if (base > point) break;
        }
        __syncthreads();
        token = found;
    }
    tell(a, b, r, j / 2, token, kThreads);
}

// ---- greedy ------------------------------------------------------------------------

// Larger values first, then lower indices; NaN least.
__device__ inline uint64_t key(float x, uint32_t i) {
    uint32_t v = __builtin_bit_cast(uint32_t, x + 0.f);  // -0 becomes 0
    v = v & 0x80000000u ? ~v : v | 0x80000000u;
    if (x != x) v = 0x007fffffu;  // that of -infinity
    return (uint64_t)v << 32 | ~i;
}

// Grid (pieces, rows).
template <int DT>
__global__ __launch_bounds__(kThreads) void k_verify_best(VerifyArgs a) {
    typedef typename Elem<DT>::type E;
    constexpr int N = Elem<DT>::kVec;
    __shared__ uint64_t part[kThreads / 64];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (row >= a.T) return;
    const E* p = static_cast<const E*>(a.p) + row * a.p_row;
    const int64_t lo = (int64_t)blockIdx.x * a.len, hi = lo + a.len < a.V ? lo + a.len : a.V;
    uint64_t best = 0;
    for (int64_t i = lo + (int64_t)tid * N; i < hi; i += (int64_t)kThreads * N) {
        if (i + N <= hi) {
            const Piece<DT> y = *reinterpret_cast<const Piece<DT>*>(p + i);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const uint64_t k = key(Elem<DT>::get(y.e[e]), (uint32_t)(i + e));
                best = k > best ? k : best;
            }
        } else {
            for (int64_t e = i; e < hi; ++e) {
                const uint64_t k = key(Elem<DT>::get(p[e]), (uint32_t)e);
                best = k > best ? k : best;
            }
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const uint64_t k = __shfl_xor((unsigned long long)best, o);
        best = k > best ? k : best;
    }
    if ((tid & 63) == 0) part[tid >> 6] = best;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int w = 1; w < kThreads / 64; ++w) best = part[w] > best ? part[w] : best;
        a.sums[row * a.pieces + blockIdx.x] = best;
    }
}

// Grid: requests; a wave a row.
__global__ __launch_bounds__(kThreads) void k_verify_first(VerifyArgs a) {
    __shared__ int least, token;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Rows r = rows_of(a, b);
    if (r.n <= 0) {
        tell(a, b, r, 0, -1, kThreads);
        return;
    }
    if (tid == 0) least = r.n - 1;
    __syncthreads();
    for (int i0 = 0;; i0 += kThreads / 64) {
        const int i = i0 + wave;
        int best = -1;
        if (i < r.n) {
            uint64_t k = 0;
            for (int c = lane; c < a.pieces; c += 64) {
                const uint64_t y = a.sums[(int64_t)(r.first + i) * a.pieces + c];
                k = y > k ? y : k;
            }
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) {
                const uint64_t y = __shfl_xor((unsigned long long)k, o);
                k = y > k ? y : k;
            }
            best = (int)~(uint32_t)k;
            if (lane == 0 && i < r.n - 1 && a.tokens[r.first + i + 1] != best) atomicMin(&least, i);
        }
        __syncthreads();
        const int j = least;
        if (i == j && lane == 0) token = best;
        __syncthreads();
        if (j < i0 + kThreads / 64) {
            tell(a, b, r, j, token, kThreads);
            return;
        }
    }
}

template <int DT>
hipError_t run(const VerifyArgs& a, hipStream_t s) {
    const int64_t rows = a.u ? a.B : a.T;
    const unsigned y = rows < 32768 ? (unsigned)rows : 32768u, z = (unsigned)((rows + y - 1) / y);
    if (a.u) k_verify_sums<DT><<<dim3((a.pieces + kWaves - 1) / kWaves, y, z), dim3(kThreads), 0, s>>>(a);
    else k_verify_best<DT><<<dim3(a.pieces, y, z), dim3(kThreads), 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.u) k_verify_pick<DT><<<dim3((unsigned)a.B), dim3(kThreads), 0, s>>>(a);
    else k_verify_first<<<dim3((unsigned)a.B), dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

int verify_pieces(int64_t rows, int64_t V, bool greedy) {
    // Workgroups for the whole card where the rows alone do not give them, of
    // 1024 elements or more.  A piece to sample from is what a wave sums and the
    // search reads: up to 2048.
    int64_t c = (1024 + rows - 1) / rows;
    const int64_t most = (V + 1023) / 1024, least = (V + 8191) / 8192;
    c = c > most ? most : c;
    c = c < least ? least : c;
    return (int)(greedy ? c : c * kWaves);
}

int64_t verify_most_pieces(int64_t rows, int64_t V, bool greedy) {
    // r rows have r ceil(1024 / r) <= r + 1023 pieces between the two limits, and a
    // piece has eight elements or is the row
    const int64_t most = (V + 1023) / 1024, least = (V + 8191) / 8192;
    int64_t n = rows + 1023 < rows * most ? rows + 1023 : rows * most;
    n = n < rows * least ? rows * least : n;
    n = greedy ? n : n * kWaves;
    const int64_t finest = rows * ((V + 7) / 8);
    return n < finest ? n : finest;
}

hipError_t launch_verify(const VerifyArgs& a, int dtype, hipStream_t s) {
    return dtype == FK_F32   ? run<FK_F32>(a, s)
           : dtype == FK_F16 ? run<FK_F16>(a, s)
                             : run<FK_BF16>(a, s);
}

}  // namespace fk
