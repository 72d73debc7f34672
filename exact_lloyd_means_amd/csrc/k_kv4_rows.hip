// k_kv4_rows.hip -- rows into the 4-bit cache and back (fk_kv4_write,
// fk_kv4_read).
//
// Sixteen lanes hold a row, D/16 consecutive dimensions each, and do its k
// and its v.
//
// Writing is bound by the comparisons unless they are few: one value meets 15
// thresholds.  A value x of the cache type and a threshold t s in fp32 compare
// as integers: with ord() the type's bits in value order, x > t s exactly
// where ord(x) > ord(the largest 16-bit value not above t s).  Lane j of the
// row finds that bound for threshold j, the row shares them through LDS, and
// two values at a time walk the search tree in packed 16-bit arithmetic (a
// saturated difference's sign is the comparison, v_bfi picks the next bound):
// 14 instructions a value, where fp32 comparisons and selects take 22.
// 16384 tokens x 8 heads x 128, k and v, 84 MB in and out: 30 us, 2.8 TB/s
// (fp32 40 us).  Reading them back is a copy: 18 us, 4.6 TB/s.
//
// A lane's codes are D/32 whole bytes of one token in both layouts, so tokens
// never share a byte and no write needs an atomic.
#include "kv4_internal.h"

#include <type_traits>

namespace fk {
namespace {

constexpr int kThreads = 256;
constexpr int kRowLanes = 16;
constexpr int kRowsPerWg = kThreads / kRowLanes;

// Where a slot lies: record index ((page * H + h) * 2) and place in the page.
struct Place {
    int64_t at;
    int in;
};
__device__ inline Place place_of(const RowArgs& a, int32_t slot, int h) {
    const uint32_t blk = (uint32_t)slot >> 5;
    const uint32_t page = a.bpp == 1 ? blk : (uint32_t)(((uint64_t)blk * a.bpp_magic) >> 32);
    return {((int64_t)page * a.H + h) * 2, (int)((uint32_t)slot - page * (uint32_t)a.page_size)};
}

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

typedef short shortx2 __attribute__((ext_vector_type(2)));

// Bits of two 16-bit floats as integers in the order of their values.
__device__ inline shortx2 ordered(uint32_t x) {
    const shortx2 v = __builtin_bit_cast(shortx2, x);
    const shortx2 sign = v >> 15;
    return v ^ (sign & (short)0x7fff);
}

// Threshold j of a codebook.
__device__ inline float threshold(const uint16_t* cb, int j) {
    const float lo = kv_f32<FK_F16>(cb[j]), hi = kv_f32<FK_F16>(cb[j < 15 ? j + 1 : 15]);
    return (float)(_Float16)(0.5f * (lo + hi));
}

// A lane's bound: the order of the largest 16-bit value not above threshold t
// times the scale, in both halves.  0x7fff, above every value, where the scale
// is NaN: code 0.
template <int DT>
__device__ inline uint32_t bound(float t, uint32_t scale) {
    const float s = kv_f32<DT>(scale);
    const float v = t * s + 0.f;  // + 0: a threshold of -0 is 0
    const uint32_t bits = kv_bits<DT>(v);
    const int o = (int)(short)(bits ^ (bits & 0x8000 ? 0x7fff : 0)) - (kv_f32<DT>(bits) > v ? 1 : 0);
    const uint32_t c = s == s ? (uint32_t)o & 0xffff : 0x7fff;
    return c | c << 16;
}

// All ones in the halves where x > c: the sign of the saturated c - x.  As
// instructions, since the compiler turns the masks back into scalar
// comparisons and selects.
__device__ inline uint32_t above(shortx2 x, uint32_t c) {
    uint32_t d;
    asm("v_pk_sub_i16 %0, %1, %2 clamp\n\tv_pk_ashrrev_i16 %0, 15, %0 op_sel_hi:[0,1]"
        : "=&v"(d)
        : "v"(c), "v"(x));
    return d;
}
__device__ inline uint32_t pick(uint32_t m, uint32_t yes, uint32_t no) {
    uint32_t d;
    asm("v_bfi_b32 %0, %1, %2, %3" : "=v"(d) : "v"(m), "v"(yes), "v"(no));
    return d;
}

// Codes of two values, in the low nibbles of the halves; c ascending.
__device__ inline uint32_t codes_of(shortx2 x, const uint32_t (&c)[16]) {
    const uint32_t m3 = above(x, c[7]);
    uint32_t u[7];
#pragma unroll
    for (int i = 0; i < 7; ++i) u[i] = pick(m3, c[8 + i], c[i]);
    const uint32_t m2 = above(x, u[3]);
    const uint32_t v0 = pick(m2, u[4], u[0]), v1 = pick(m2, u[5], u[1]), v2 = pick(m2, u[6], u[2]);
    const uint32_t m1 = above(x, v1);
    const uint32_t m0 = above(x, pick(m1, v2, v0));
    return (m3 & 0x00080008) | (m2 & 0x00040004) | (m1 & 0x00020002) | (m0 & 0x00010001);
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

// Codes of a lane's D/16 values as D/32 bytes and the row's scale bits.  row:
// 16 words of LDS of this row.
template <int D, int DT>
__device__ inline void encode(const uint32_t (&x)[D / 32], float t, uint32_t* row, int r,
                              uint32_t& scale, uint64_t& bytes) {
    uint32_t m = x[0] & 0x7fff7fff;
#pragma unroll
    for (int i = 1; i < D / 32; ++i) m = max_u16(m, x[i] & 0x7fff7fff);
    m = row_max(m >> 16 > (m & 0xffff) ? m >> 16 : m & 0xffff);
    constexpr uint32_t inf = DT == FK_BF16 ? 0x7f80 : 0x7c00, nan = DT == FK_BF16 ? 0x7fc0 : 0x7e00;
    scale = m >= inf ? nan : m;
    row[r] = bound<DT>(t, scale);
    // the row's lanes are of one wave: no barrier, but the reads stay behind the writes
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    uint32_t c[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 y = reinterpret_cast<const uint4*>(row)[i];
        c[4 * i] = y.x;
        c[4 * i + 1] = y.y;
        c[4 * i + 2] = y.z;
        c[4 * i + 3] = y.w;
    }
    bytes = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const uint32_t y = codes_of(ordered(x[i]), c);
        bytes |= (uint64_t)((y | y >> 12) & 0xff) << (8 * i);
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
    __shared__ uint32_t bounds[2][kRowsPerWg][16];
    const int tid = threadIdx.x, r = tid & 15;
    uint32_t *kc = bounds[0][tid >> 4], *vc = bounds[1][tid >> 4];
    const int group = blockIdx.x / (uint32_t)a.H, h = blockIdx.x - group * a.H;
    const int tok = group * kRowsPerWg + (tid >> 4);
    if (tok >= a.T) return;
    uint32_t x[D / 32], y[D / 32];
    load_row<D, DT, VEC>(a.k + tok * a.k_token + h * a.k_head + r * (D / 16), x);
    load_row<D, DT, VEC>(a.v + tok * a.v_token + h * a.v_head + r * (D / 16), y);
    const int32_t slot = a.slots[tok];
    const float tk = threshold(a.codebook + h * 16, r), tv = threshold(a.codebook + (a.H + h) * 16, r);
    if (slot < 0 || slot >= a.slots_total) return;  // the same for the whole row's lanes
    const Place p = place_of(a, slot, h);
    const int i = p.in & 31;
    uint8_t* kb = a.codes + (p.at * a.bpp + (p.in >> 5)) * (16 * D);
    uint8_t* vb = kb + a.bpp * (16 * D);
    uint16_t* sc = a.scales + p.at * a.page_size + p.in;
    uint32_t s;
    uint64_t b;
    encode<D, DT>(x, tk, kc, r, s, b);
    store_bytes<D>(kb + k_place<D>(i, r), b);
    if (r == 0) sc[0] = (uint16_t)s;
    encode<D, DT>(y, tv, vc, r, s, b);
    if constexpr (D == 256) {
        *reinterpret_cast<uint32_t*>(vb + v_place<D>(i, r, 0)) = (uint32_t)b;
        *reinterpret_cast<uint32_t*>(vb + v_place<D>(i, r, 1)) = (uint32_t)(b >> 32);
    } else {
        store_bytes<D>(vb + v_place<D>(i, r, 0), b);
    }
    if (r == 0) sc[a.page_size] = (uint16_t)s;
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
    __shared__ float cb[2][16];
    const int tid = threadIdx.x, r = tid & 15;
    const int group = blockIdx.x / (uint32_t)a.H, h = blockIdx.x - group * a.H;
    if (tid < 32) cb[tid >> 4][tid & 15] = kv_f32<FK_F16>(a.codebook[((tid >> 4) * a.H + h) * 16 + (tid & 15)]);
    __syncthreads();
    const int tok = group * kRowsPerWg + (tid >> 4);
    if (tok >= a.T) return;
    const int32_t slot = a.slots[tok];
    const bool there = slot >= 0 && slot < a.slots_total;
    const Place p = place_of(a, there ? slot : 0, h);
    const int64_t at = p.at;
    const int in = p.in;
    const int64_t plane = (int64_t)a.bpp * (16 * D);
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
    const int64_t o = ((int64_t)tok * a.H + h) * D + r * (D / 16);
    decode<D, DT>(k, ks, cb[0], a.ko + o);
    decode<D, DT>(v, vs, cb[1], a.vo + o);
}

// Sixteen tokens of one head a workgroup, so that neighbours in a page fill
// whole lines of its blocks; the heads of the same tokens next to each other,
// since their rows are neighbours in k and v.
dim3 row_grid(const RowArgs& a) {
    return dim3((unsigned)((a.T + kRowsPerWg - 1) / kRowsPerWg * a.H));
}

template <int D, int DT>
hipError_t write_as(const RowArgs& a, bool vec, hipStream_t s) {
    auto kern = vec ? k_kv4_write<D, DT, true> : k_kv4_write<D, DT, false>;
    kern<<<row_grid(a), dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
}

template <int D, int DT>
hipError_t read_as(const RowArgs& a, hipStream_t s) {
    k_kv4_read<D, DT><<<row_grid(a), dim3(kThreads), 0, s>>>(a);
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
