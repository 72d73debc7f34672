// k_rope.hip -- rotary positions of rows of heads (fk_rope).
//
// Pair i of a token at position p turns by p turns_i.  The product of the
// 32-bit position and the 64-bit fraction of a turn is taken modulo 2^64, that
// is modulo a turn, so the angle is exact to 2^-33 turn for every position
// (in fp32 a position of 2^17 alone leaves 2^-7 radian).  Its top bits give
// the quadrant, the rest an angle within an eighth of a turn, where the Taylor
// series of sine (to x^9) and cosine (to x^10) are off by less than 3e-9.
//
// Bound by memory: read and written once.  A thread keeps the sines of its
// pairs and walks the heads; threads of a row lie side by side and rows of
// neighbouring heads behind them, so that a wave reads 2 KB in one piece.  16384
// tokens x 40 heads of 128 bf16: 71 us, 4.7 TB/s, what a copy reaches; 64
// tokens: 3.6 us, a launch and two dependent reads.  5001 tokens x 9 heads of 64
// fp32, half rotated: 8.0 us (memory alone 4.9), since eight heads are walked at
// once and the ninth takes a round of its own.
#include "serve_internal.h"

namespace fk {
namespace {

__device__ inline void sincos_turn(uint64_t phase, float& s, float& c) {
    const uint32_t t = (uint32_t)((phase + 0x80000000u) >> 32);
    const uint32_t quad = (t + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(t - (quad << 30)) * 1.46291807926715968e-9f;  // 2 pi / 2^32
    const float y = x * x;
    const float sn = x + x * y * (-1.f / 6 + y * (1.f / 120 + y * (-1.f / 5040 + y * (1.f / 362880))));
    const float cs = 1.f + y * (-0.5f + y * (1.f / 24 + y * (-1.f / 720 + y * (1.f / 40320 +
                                                                              y * (-1.f / 3628800)))));
    const bool swap = quad & 1;
    s = swap ? cs : sn;
    c = swap ? sn : cs;
    s = quad & 2 ? -s : s;
    c = (quad + 1) & 2 ? -c : c;
}

template <int DT>
struct Elem {
    typedef uint16_t type;
    static constexpr int kVec = 8;
};
template <>
struct Elem<FK_F32> {
    typedef float type;
    static constexpr int kVec = 4;
};

template <int DT>
__device__ inline float to_f32(typename Elem<DT>::type x) {
    if constexpr (DT == FK_F32) return x;
    else return kv_f32<DT>(x);
}
template <int DT>
__device__ inline typename Elem<DT>::type from_f32(float x) {
    if constexpr (DT == FK_F32) return x;
    else return (uint16_t)kv_bits<DT>(x);
}

template <typename E, int N>
struct alignas(sizeof(E) * N) Pack {
    E e[N];
};

// Threads (unit of a row, head, token).  With VEC a unit is 16 bytes of the
// row (interleaved) or 16 bytes of each half; otherwise a pair.  Units behind
// the rotated part copy what is left of the row.
template <int DT, bool INTER, bool VEC>
__global__ __launch_bounds__(256) void k_rope(RopeArgs a) {
    typedef typename Elem<DT>::type E;
    constexpr int N = VEC ? Elem<DT>::kVec : 1;     // elements of an access
    constexpr int kPairs = INTER ? (VEC ? N / 2 : 1) : N;
    const int64_t tok = (int64_t)blockIdx.x * blockDim.z + threadIdx.z;
    if (tok >= a.T) return;
    const int u = threadIdx.x + blockIdx.z * blockDim.x;
    if (u >= a.units) return;
    const int head0 = threadIdx.y + blockIdx.y * blockDim.y, step = blockDim.y * gridDim.y;
    const int p = a.pos[tok];
    const bool turn = u < a.turn_units && p >= 0;
    // first element of the unit, and of its other half
    const int at = u < a.turn_units ? u * (INTER ? kPairs * 2 : N) : a.R + (u - a.turn_units) * N;
    const int second = INTER ? (VEC ? at : at + 1) : at + a.R / 2;
    const bool two = u < a.turn_units && second != at;
    float s[kPairs], c[kPairs];
    if (turn) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            sincos_turn((uint64_t)(uint32_t)p * a.turns[u * kPairs + i], s[i], c[i]);
            s[i] *= a.sin_factor;
            c[i] *= a.factor;
        }
    }
    for (int h = head0; h < a.heads[0] + a.heads[1]; h += step) {
        const int w = h >= a.heads[0], hh = w ? h - a.heads[0] : h;
        const RopeSet& r = a.set[w];
        if (!turn && r.x == r.y) continue;
        typedef Pack<E, N> V;
        const E* x = static_cast<const E*>(r.x) + tok * r.x_token + hh * r.x_head;
        E* y = static_cast<E*>(r.y) + tok * r.y_token + hh * r.y_head;
        V lo = *reinterpret_cast<const V*>(x + at), hi;
        if (two) hi = *reinterpret_cast<const V*>(x + second);
        if (turn) {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                constexpr bool in_one = INTER && VEC;
                E& ea = in_one ? lo.e[2 * i] : lo.e[i];
                E& eb = in_one ? lo.e[(2 * i + 1) % N] : hi.e[i];
                const float xa = to_f32<DT>(ea), xb = to_f32<DT>(eb);
                ea = from_f32<DT>(xa * c[i] - xb * s[i]);
                eb = from_f32<DT>(xb * c[i] + xa * s[i]);
            }
        }
        *reinterpret_cast<V*>(y + at) = lo;
        if (two) *reinterpret_cast<V*>(y + second) = hi;
    }
}

template <int DT, bool INTER>
void launch(const RopeArgs& a, bool vec, dim3 grid, dim3 block, hipStream_t s) {
    if (vec) k_rope<DT, INTER, true><<<grid, block, 0, s>>>(a);
    else k_rope<DT, INTER, false><<<grid, block, 0, s>>>(a);
}

template <int DT>
hipError_t launch_dt(RopeArgs a, bool inter, hipStream_t s) {
    constexpr int N = Elem<DT>::kVec;
    // 16-byte accesses where every row and both halves start on 16 bytes
    bool vec = inter ? a.R % N == 0 : a.R / 2 % N == 0;
    vec = vec && a.D % N == 0;
    for (const RopeSet& r : a.set)
        vec = vec && !((reinterpret_cast<uintptr_t>(r.x) | reinterpret_cast<uintptr_t>(r.y)) & 15) &&
              !((r.x_token | r.x_head | r.y_token | r.y_head) % N);
    const int pairs = inter ? (vec ? N / 2 : 1) : (vec ? N : 1);
    a.turn_units = a.R / 2 / pairs;
    a.units = a.turn_units + (a.D - a.R) / (vec ? N : 1);
    const int heads = a.heads[0] + a.heads[1];
    // a launch has less than 2^32 threads in a dimension, and up to 2^24 tokens
    const int most = a.T > 1 << 23 ? 128 : 256, x = a.units < most ? a.units : most;
    int y = 256 / x < heads ? 256 / x : heads;
    // Heads walked by a thread share its sines; few tokens have them spread
    // over more workgroups instead, until about eight waves a SIMD are there.
    const int64_t threads = a.T * a.units;
    int64_t lanes = (int64_t)256 * 4 * 8 * 64 / (threads < 1 ? 1 : threads);  // heads at once
    lanes = lanes < 1 ? 1 : lanes > heads ? heads : lanes;
    if (y > 8 && lanes < y) y = lanes < 8 ? 8 : (int)lanes;
    const int gy = (int)((lanes + y - 1) / y);
    int z = 256 / (x * y);
    z = z < 1 ? 1 : z > 64 ? 64 : z;
    const dim3 block(x, y, z), grid((unsigned)((a.T + z - 1) / z), gy, (a.units + x - 1) / x);
    if (inter) launch<DT, true>(a, vec, grid, block, s);
    else launch<DT, false>(a, vec, grid, block, s);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, int dtype, bool inter, hipStream_t s) {
    return dtype == FK_F32   ? launch_dt<FK_F32>(a, inter, s)
           : dtype == FK_F16 ? launch_dt<FK_F16>(a, inter, s)
                             : launch_dt<FK_BF16>(a, inter, s);
}

}  // namespace fk
