// k_kv4_rows.hip -- rows into the 4-bit cache and back (fk_kv4_write,
// fk_kv4_read).
//
// Sixteen lanes hold a row, D/16 consecutive dimensions each, and do its k
// and its v.  Writing: s = max |x| over the row (an integer maximum of the
// bits without sign, which also finds NaN and infinities), thresholds t_j s,
// and each value's code by four comparisons of a search tree held in
// registers.  A lane's codes are D/32 whole bytes of one token in both
// layouts, so tokens never share a byte and no write needs an atomic.
#include "kv4_internal.h"

#include <type_traits>

namespace fk {
namespace {

constexpr int kThreads = 256;
constexpr int kRowLanes = 16;
constexpr int kRowsPerWg = kThreads / kRowLanes;

// Byte offset of lane r's D/32 bytes of token t in its k block.
template <int D>
__device__ inline int k_place(int t, int r) {
    const int m = 4 * (t >> 3) + (t & 3), tile = (t >> 2) & 1;
    const int a = tile * (D / 8) + (r & 3) * (D / 32);
    return (a >> 4) * 1024 + (16 * (r >> 2) + m) * 16 + (a & 15);
}
// The same in its v block; piece `half` of 4 bytes for D = 256.
template <int D>
__device__ inline int v_place(int t, int r, int half) {
    constexpr int w = D / 32 < 4 ? D / 32 : 4;
    const int a = half * 32 + (t & 7) * w;
    return (a >> 4) * 1024 + (16 * (t >> 3) + r) * 16 + (a & 15);
}

// Maximum over the 16 lanes of a row.
__device__ inline uint32_t row_max(uint32_t x) {
    auto step = [&](auto ctrl) {
        const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value,
                                                                 0xf, 0xf, false);
        x = x > y ? x : y;
    };
    step(std::integral_constant<int, 0x128>{});  // rotations by 8, 4, 2, 1
    step(std::integral_constant<int, 0x124>{});
    step(std::integral_constant<int, 0x122>{});
    step(std::integral_constant<int, 0x121>{});
    return x;
}

// Number of thresholds below x; t ascending.
__device__ inline uint32_t code_of(float x, const float (&t)[15]) {
    const bool c3 = t[7] < x;
    float u[7];
#pragma unroll
    for (int i = 0; i < 7; ++i) u[i] = c3 ? t[8 + i] : t[i];
    const bool c2 = u[3] < x;
    const float v0 = c2 ? u[4] : u[0], v1 = c2 ? u[5] : u[1], v2 = c2 ? u[6] : u[2];
    const bool c1 = v1 < x;
    const float w = c1 ? v2 : v0;
    return (c3 ? 8u : 0u) | (c2 ? 4u : 0u) | (c1 ? 2u : 0u) | (w < x ? 1u : 0u);
}

template <int D, int DT, bool VEC>
__device__ inline void load_row(const uint16_t* p, uint32_t (&x)[D / 32]) {
    if constexpr (VEC) {
        if constexpr (D == 64) {
            const uint2 y = *reinterpret_cast<const uint2*>(p);
            x[0] = y.x;
            x[1] = y.y;
        } else {
#pragma unroll
            for (int i = 0; i < D / 128; ++i) {
                const uint4 y = reinterpret_cast<const uint4*>(p)[i];
                x[4 * i] = y.x;
                x[4 * i + 1] = y.y;
                x[4 * i + 2] = y.z;
                x[4 * i + 3] = y.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) x[i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
    }
}

// Codes of a lane's D/16 values as D/32 bytes and the row's scale bits.
template <int D, int DT>
__device__ inline void encode(const uint32_t (&x)[D / 32], const float* thr, uint32_t& scale,
                              uint64_t& bytes) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const uint32_t lo = x[i] & 0x7fff, hi = (x[i] >> 16) & 0x7fff;
        m = m > lo ? m : lo;
        m = m > hi ? m : hi;
    }
    m = row_max(m);
    constexpr uint32_t inf = DT == FK_BF16 ? 0x7f80 : 0x7c00, nan = DT == FK_BF16 ? 0x7fc0 : 0x7e00;
    scale = m >= inf ? nan : m;
    const float s = kv_f32<DT>(scale);
    float t[15];
#pragma unroll
    for (int j = 0; j < 15; ++j) t[j] = thr[j] * s;
    bytes = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const uint32_t b = code_of(kv_f32<DT>(x[i] & 0xffff), t) |
                           code_of(kv_f32<DT>(x[i] >> 16), t) << 4;
        bytes |= (uint64_t)b << (8 * i);
    }
}

// Thresholds of the codebooks into LDS, [kv][H][16].
__device__ inline void load_thresholds(const uint16_t* cb, float* thr, int H, int tid) {
    for (int i = tid; i < 2 * H * 16; i += kThreads) {
        const float lo = kv_f32<FK_F16>(cb[i]);
        const float hi = (i & 15) < 15 ? kv_f32<FK_F16>(cb[i + 1]) : lo;
        thr[i] = (float)(_Float16)(0.5f * (lo + hi));
    }
}

template <int D>
__device__ inline void store_bytes(uint8_t* p, uint64_t b) {
    if constexpr (D == 64) *reinterpret_cast<uint16_t*>(p) = (uint16_t)b;
    else if constexpr (D == 128) *reinterpret_cast<uint32_t*>(p) = (uint32_t)b;
    else *reinterpret_cast<uint64_t*>(p) = b;
}

template <int D, int DT, bool VEC>
__global__ __launch_bounds__(kThreads) void k_kv4_write(RowArgs a) {
    extern __shared__ float thr[];
    const int tid = threadIdx.x, r = tid & 15;
    load_thresholds(a.codebook, thr, a.H, tid);
    __syncthreads();
    const int64_t rows = a.T * a.H;
    for (int64_t row = (int64_t)blockIdx.x * kRowsPerWg + (tid >> 4); row < rows;
         row += (int64_t)gridDim.x * kRowsPerWg) {
        const int64_t tok = row / a.H;
        const int h = (int)(row - tok * a.H);
        const int32_t slot = a.slots[tok];
        if (slot < 0 || slot >= a.slots_total) continue;  // the whole row's lanes
        uint32_t x[D / 32], y[D / 32];
        load_row<D, DT, VEC>(a.k + tok * a.k_token + h * a.k_head + r * (D / 16), x);
        load_row<D, DT, VEC>(a.v + tok * a.v_token + h * a.v_head + r * (D / 16), y);
        const int32_t page = (uint32_t)slot / (uint32_t)a.page_size;
        const int in = slot - page * a.page_size;
        const int64_t at = ((int64_t)page * a.H + h) * 2;
        const int64_t plane = (int64_t)a.page_size / kKvBlock * (16 * D);
        uint8_t* kb = a.codes + at * plane + (int64_t)(in >> 5) * (16 * D);
        uint8_t* vb = kb + plane;
        uint32_t s;
        uint64_t b;
        encode<D, DT>(x, thr + h * 16, s, b);
        store_bytes<D>(kb + k_place<D>(in & 31, r), b);
        if (r == 0) a.scales[at * a.page_size + in] = (uint16_t)s;
        encode<D, DT>(y, thr + (a.H + h) * 16, s, b);
        if constexpr (D == 256) {
            *reinterpret_cast<uint32_t*>(vb + v_place<D>(in & 31, r, 0)) = (uint32_t)b;
            *reinterpret_cast<uint32_t*>(vb + v_place<D>(in & 31, r, 1)) = (uint32_t)(b >> 32);
        } else {
            store_bytes<D>(vb + v_place<D>(in & 31, r, 0), b);
        }
        if (r == 0) a.scales[(at + 1) * a.page_size + in] = (uint16_t)s;
    }
}

template <int D>
__device__ inline uint64_t load_bytes(const uint8_t* p) {
    if constexpr (D == 64) return *reinterpret_cast<const uint16_t*>(p);
    else if constexpr (D == 128) return *reinterpret_cast<const uint32_t*>(p);
    else return *reinterpret_cast<const uint64_t*>(p);
}

// D/16 values of a lane, rounded once, to global memory.
template <int D, int DT>
__device__ inline void decode(uint64_t b, float s, const float* cb, uint16_t* out) {
    uint32_t y[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const uint32_t c = (uint32_t)(b >> (8 * i));
        y[i] = kv_bits<DT>(cb[c & 15] * s) | kv_bits<DT>(cb[(c >> 4) & 15] * s) << 16;
    }
    if constexpr (D == 64) {
        *reinterpret_cast<uint2*>(out) = make_uint2(y[0], y[1]);
    } else {
#pragma unroll
        for (int i = 0; i < D / 128; ++i)
            reinterpret_cast<uint4*>(out)[i] =
                make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
    }
}

template <int D, int DT>
__global__ __launch_bounds__(kThreads) void k_kv4_read(RowArgs a) {
    extern __shared__ float cb[];  // [kv][H][16]
    const int tid = threadIdx.x, r = tid & 15;
    for (int i = tid; i < 2 * a.H * 16; i += kThreads) cb[i] = kv_f32<FK_F16>(a.codebook[i]);
    __syncthreads();
    const int64_t rows = a.T * a.H;
    for (int64_t row = (int64_t)blockIdx.x * kRowsPerWg + (tid >> 4); row < rows;
         row += (int64_t)gridDim.x * kRowsPerWg) {
        const int64_t tok = row / a.H;
        const int h = (int)(row - tok * a.H);
        const int32_t slot = a.slots[tok];
        const bool there = slot >= 0 && slot < a.slots_total;
        const int32_t page = there ? (uint32_t)slot / (uint32_t)a.page_size : 0;
        const int in = there ? slot - page * a.page_size : 0;
        const int64_t at = ((int64_t)page * a.H + h) * 2;
        const int64_t plane = (int64_t)a.page_size / kKvBlock * (16 * D);
        const uint8_t* kb = a.codes + at * plane + (int64_t)(in >> 5) * (16 * D);
        const uint8_t* vb = kb + plane;
        const uint64_t k = load_bytes<D>(kb + k_place<D>(in & 31, r));
        uint64_t v;
        if constexpr (D == 256)
            v = *reinterpret_cast<const uint32_t*>(vb + v_place<D>(in & 31, r, 0)) |
                (uint64_t) * reinterpret_cast<const uint32_t*>(vb + v_place<D>(in & 31, r, 1)) << 32;
        else
            v = load_bytes<D>(vb + v_place<D>(in & 31, r, 0));
        const float ks = there ? kv_f32<DT>(a.scales[at * a.page_size + in]) : 0.f;
        const float vs = there ? kv_f32<DT>(a.scales[(at + 1) * a.page_size + in]) : 0.f;
        const int64_t o = row * D + r * (D / 16);
        decode<D, DT>(k, ks, cb + h * 16, a.ko + o);
        decode<D, DT>(v, vs, cb + (a.H + h) * 16, a.vo + o);
    }
}

unsigned row_wgs(const RowArgs& a) {
    const int64_t wgs = (a.T * a.H + kRowsPerWg - 1) / kRowsPerWg;
    return (unsigned)(wgs > (1 << 20) ? (1 << 20) : wgs);
}

template <int D, int DT>
hipError_t write_as(const RowArgs& a, bool vec, hipStream_t s) {
    const unsigned lds = 2u * a.H * 16 * 4;
    auto kern = vec ? k_kv4_write<D, DT, true> : k_kv4_write<D, DT, false>;
    static LdsAttr rec[2];
    if (lds > 65536) {
        hipError_t e = ensure_lds(rec[vec], reinterpret_cast<const void*>(kern), 131072);
        if (e != hipSuccess) return e;
    }
    kern<<<dim3(row_wgs(a)), dim3(kThreads), lds, s>>>(a);
    return hipGetLastError();
}

template <int D, int DT>
hipError_t read_as(const RowArgs& a, hipStream_t s) {
    const unsigned lds = 2u * a.H * 16 * 4;
    static LdsAttr rec;
    if (lds > 65536) {
        hipError_t e = ensure_lds(rec, reinterpret_cast<const void*>(k_kv4_read<D, DT>), 131072);
        if (e != hipSuccess) return e;
    }
    k_kv4_read<D, DT><<<dim3(row_wgs(a)), dim3(kThreads), lds, s>>>(a);
    return hipGetLastError();
}

template <int D>
hipError_t write_d(const RowArgs& a, int dtype, bool vec, hipStream_t s) {
    return dtype == FK_BF16 ? write_as<D, FK_BF16>(a, vec, s) : write_as<D, FK_F16>(a, vec, s);
}
template <int D>
hipError_t read_d(const RowArgs& a, int dtype, hipStream_t s) {
    return dtype == FK_BF16 ? read_as<D, FK_BF16>(a, s) : read_as<D, FK_F16>(a, s);
}

}  // namespace

hipError_t launch_kv4_write(const RowArgs& a, int D, int dtype, bool vec, hipStream_t s) {
    return D == 64 ? write_d<64>(a, dtype, vec, s)
                   : D == 128 ? write_d<128>(a, dtype, vec, s) : write_d<256>(a, dtype, vec, s);
}

hipError_t launch_kv4_read(const RowArgs& a, int D, int dtype, hipStream_t s) {
    return D == 64 ? read_d<64>(a, dtype, s)
                   : D == 128 ? read_d<128>(a, dtype, s) : read_d<256>(a, dtype, s);
}

}  // namespace fk
