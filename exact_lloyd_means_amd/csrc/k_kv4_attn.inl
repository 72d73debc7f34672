// k_kv4_attn.inl -- attention over the 4-bit paged cache (fk_kv4_attention).
//
// One wave holds 16 NT query rows and walks blocks of 32 cached tokens:
//
//   S^T = K Q^T   v_mfma_f32_16x16x32_f16, A = 16 tokens x 32 dimensions of
//                 codebook values, B = 32 dimensions x 16 query rows.  Lane
//                 (16 g + n) gets rows 4 g + r of query n.  The token of row
//                 m of tile u is 8 (m / 4) + 4 u + m % 4, so the two tiles
//                 give a lane the eight consecutive tokens 8 g .. 8 g + 7.
//   p, w          x = S * (k scale * scale log2 e), p = 2^(x qs - m), l += p,
//                 w = p * v scale, all in fp32 in those lanes; w rounded to
//                 fp16 once.  qs is a power of two, so x qs is exact and the
//                 largest scores cancel in x qs - m however large they are.
//   O^T += V^T w  A = 16 dimensions x 32 tokens, B = w: a lane's operand is
//                 its own eight weights, so nothing crosses lanes.
//
// The rows of a (request, kv head) are numbered token * G + head of the
// group: all query heads of a group and a few tokens share one pass.
//
// Codes become fp16 through a table in LDS of all 256 pairs of codebook
// values, one 4-byte entry per byte of codes: k's at 256 byte, v's 128 bytes
// on, each 32 times side by side so that the 32 lanes read at once lie in 32
// banks whatever their codes.  The address (byte << 8 | 4 (lane % 32)) is one
// v_perm of the codes.  (16-entry tables in registers cost 11 v_perm and
// masks per 4 values; this costs 2 and 2 LDS reads.)  k's codes come in
// operand order.  A lane's v codes are an 8 x 8 tile (token, dimension) of
// nibbles that is transposed in registers, half an instruction a value.
//
// m follows what a row adds up, not its scores alone: it is 3 below the log2 of
// the row's largest p * v scale when it is set, and is raised only when a
// weight could pass 2^15, so that most blocks need no reduction over lanes and
// no rescaling.  A row's largest weight is therefore 8 or more, all are in
// fp16's range, and rounding costs a weight 2^-11 of itself or 2^-28 of the
// row's largest, whatever the scales of tokens that the row hardly counts or
// does not see.  m scales O and l alike and cancels; l is summed over lanes at
// the end, in fp32.
#pragma once

#include "kv4_internal.h"

namespace fk {
namespace {

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = 4;
constexpr int kTabBytes = 65536;
constexpr int kSplitLds = kTabBytes + 512;  // and what the waves tell each other
constexpr float kNoMax = -3.402823466e38f;  // m before any key: below every score
constexpr float kFirst = 3.f;      // log2 of a row's largest weight when m is set
constexpr float kRoom = 4.f;       // log2 of the room above a block's largest v scale
constexpr float kTop = 15.f;       // log2 of the largest weight
// v scales below 2^-93 count as that in m, and no p passes 2^96.5, so that l
// stays finite over 2^31 tokens whose v is zero.
constexpr float kLeastScale = -93.f, kMostP = 96.5f;

typedef uint32_t uintx4 __attribute__((ext_vector_type(4)));

struct Rows {       // the query rows of a tile within their request
    int qlen, seq;  // of the request
    int tok0;       // its first query token
    int r0, n;      // first row, number of rows
};

// Blocks [lo, hi) that some row of the tile sees.
struct Span {
    int lo, hi;
};

// x / y for x < 2^24 with magic = ceil(2^32 / y), y <= 256.
__device__ inline int divide(int x, uint32_t y, uint32_t magic) {
    return y == 1 ? x : (int)(((uint64_t)(uint32_t)x * magic) >> 32);
}

__device__ inline void request_lens(const AttnArgs& a, int b, Rows& rw) {
    const int T = (int)a.T;
    int c0 = a.cu[b], c1 = a.cu[b + 1];
    const int s = a.seq[b];
    c0 = c0 < 0 ? 0 : c0 > T ? T : c0;
    c1 = c1 < c0 ? c0 : c1 > T ? T : c1;
    rw.tok0 = c0;
    rw.qlen = c1 - c0;
    rw.seq = s < 0 ? 0 : s;
}

// First and one past the last position that query token i sees.
__device__ inline void bounds(const AttnArgs& a, const Rows& rw, int i, int& lo, int& hi) {
    const int pos = rw.seq - rw.qlen + i;
    hi = a.causal ? pos + 1 : rw.seq;
    hi = hi > a.cap ? a.cap : hi;
    hi = hi < 0 ? 0 : hi;
    lo = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
    lo = lo > hi ? hi : lo;
}

// Rows r0 .. of the request in tiles of `rows`, and the blocks they see.  Query
// tokens from max_q on have no rows: tiles and workspace are laid out for max_q,
// and what cu says is only known here.
__device__ inline Span tile_rows(const AttnArgs& a, Rows& rw, int r0, int rows) {
    rw.r0 = r0;
    const int left = (rw.qlen < a.max_q ? rw.qlen : a.max_q) * a.G - r0;
    rw.n = left < 0 ? 0 : left > rows ? rows : left;
    if (rw.n <= 0) return {0, 0};
    int lo, hi, t0, t1;
    bounds(a, rw, divide(r0, a.G, a.G_magic), lo, t0);
    bounds(a, rw, divide(r0 + rw.n - 1, a.G, a.G_magic), t1, hi);
    if (hi <= lo) return {0, 0};
    return {lo / kKvBlock, (hi + kKvBlock - 1) / kKvBlock};
}

__device__ inline floatx4 mfma(half8 x, half8 y, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, c, 0, 0, 0);
}

// The table starts the workgroup's LDS (the kernels have no static LDS), so an
// entry's address needs no base.
typedef const __attribute__((address_space(3))) uint32_t* LdsWord;

// Eight codes of a dword to eight fp16 codebook values.  lane4 = 4 (lane %
// 32) selects the lane's copy of the table, V the codebook.
template <bool V>
__device__ inline half8 lookup(uint32_t codes, uint32_t lane4) {
    uintx4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // bytes of the address: lane4's byte 0, byte i of the codes, zeros
        const uint32_t at = __builtin_amdgcn_perm(codes, lane4, 0x0c0c0000u | (4u + i) << 8);
        y[i] = *((LdsWord)(uintptr_t)at + (V ? 32 : 0));
    }
    return __builtin_bit_cast(half8, y);
}

// The pair table of one kv head: 256 entries of 64 dwords, k copies in 0-31,
// v copies in 32-63.  A thread writes the 16-byte column tid % 16 of entries
// whose low nibble is tid / 16 % 16.
__device__ inline void build_table(uint32_t* tab, const uint16_t* codebook, int H, int h, int tid,
                                   int threads) {
    const int col = tid & 15, lo = tid >> 4 & 15;
    const uint16_t* cb = codebook + ((col >> 3) * H + h) * 16;
    const uint32_t low = cb[lo];
    for (int i = tid >> 8; i < 16; i += threads >> 8) {
        const uint32_t v = low | (uint32_t)cb[i] << 16;
        uintx4 y = {v, v, v, v};
        *reinterpret_cast<uintx4*>(tab + (i * 16 + lo) * 64 + col * 4) = y;
    }
}

// 8 rows (tokens) x 8 columns (dimensions) of nibbles, one row a dword, to 8
// columns of 8 rows.
__device__ inline void pair_columns(uint32_t even, uint32_t odd, uint32_t& c0, uint32_t& c1) {
    constexpr uint32_t m = 0x0f0f0f0fu;
    c0 = (even & m) | ((odd << 4) & ~m);
    c1 = ((even >> 4) & m) | (odd & ~m);
}
__device__ inline void transpose8(const uint32_t (&x)[8], uint32_t (&y)[8]) {
    uint32_t a[4], b[4];  // columns 0-3, 4-7 of rows j and j + 4
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        a[j] = __builtin_amdgcn_perm(x[j + 4], x[j], 0x05040100u);
        b[j] = __builtin_amdgcn_perm(x[j + 4], x[j], 0x07060302u);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const uint32_t* s = c ? b : a;
        const uint32_t lo0 = __builtin_amdgcn_perm(s[2], s[0], 0x06020400u);
        const uint32_t lo1 = __builtin_amdgcn_perm(s[3], s[1], 0x06020400u);
        const uint32_t hi0 = __builtin_amdgcn_perm(s[2], s[0], 0x07030501u);
        const uint32_t hi1 = __builtin_amdgcn_perm(s[3], s[1], 0x07030501u);
        pair_columns(lo0, lo1, y[4 * c], y[4 * c + 1]);
        pair_columns(hi0, hi1, y[4 * c + 2], y[4 * c + 3]);
    }
}
// 8 rows x 4 columns, two rows a dword.
__device__ inline void transpose4(const uint32_t (&x)[4], uint32_t (&y)[4]) {
    // bytes 0, 1 of a dword: columns 0-1, 2-3 of an even row; 2, 3: of the odd row
    const uint32_t e0 = __builtin_amdgcn_perm(x[1], x[0], 0x05010400u);  // even rows 0, 2: c01 c01 c23 c23
    const uint32_t e1 = __builtin_amdgcn_perm(x[3], x[2], 0x05010400u);
    const uint32_t o0 = __builtin_amdgcn_perm(x[1], x[0], 0x07030602u);
    const uint32_t o1 = __builtin_amdgcn_perm(x[3], x[2], 0x07030602u);
    pair_columns(__builtin_amdgcn_perm(e1, e0, 0x05040100u),
                 __builtin_amdgcn_perm(o1, o0, 0x05040100u), y[0], y[1]);
    pair_columns(__builtin_amdgcn_perm(e1, e0, 0x07060302u),
                 __builtin_amdgcn_perm(o1, o0, 0x07060302u), y[2], y[3]);
}

// Maxima that skip the quieting of NaN operands that fmaxf comes with; a NaN
// loses to a number.
__device__ inline float max2(float x, float y) {
    float r;
    asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(x), "v"(y));
    return r;
}
__device__ inline float max3(float x, float y, float z) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(x), "v"(y), "v"(z));
    return r;
}

// 2^e as bits of the cache dtype in both halves, at most infinity's.
template <int DT>
__device__ inline uint32_t pow2_bits(int e) {
    uint32_t b;
    if constexpr (DT == FK_BF16) b = (uint32_t)(e + 127) << 7;
    else b = e < -14 ? 1u << (e + 24) : (uint32_t)(e + 15) << 10;
    const uint32_t inf = DT == FK_BF16 ? 0x7f80 : 0x7c00;
    b = b < inf ? b : inf;
    return b | b << 16;
}

// The halves of a dword of scales as fp32.  For fp16 by instruction: left to
// itself the compiler folds the conversions into mixed-precision products and
// pays with registers that the accumulators need.
template <int DT>
__device__ inline float low_f32(uint32_t x) {
    if constexpr (DT == FK_BF16) return __builtin_bit_cast(float, x << 16);
    float r;
    asm("v_cvt_f32_f16_e32 %0, %1" : "=v"(r) : "v"(x));
    return r;
}
template <int DT>
__device__ inline float high_f32(uint32_t x) {
    if constexpr (DT == FK_BF16) return __builtin_bit_cast(float, x & 0xffff0000u);
    float r;
    asm("v_cvt_f32_f16_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:WORD_1"
        : "=v"(r) : "v"(x));
    return r;
}

__device__ inline float max_groups(float x) {  // over the four lanes of a query row
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}

// Where a lane reads a block: its first codes of k and v, its scales.
struct Source {
    const uint8_t *k, *v;
    const uint16_t *ks, *vs;
    bool there;
};

// The codes and scales of one block, as one lane reads them.
template <int D>
struct Block {
    uintx4 k[D / 64], v[D / 64], ks, vs;
    bool there;

    // Both scales come with k's codes: the weights need them, and waiting for the
    // last load of a block would be waiting for v's codes, a softmax too early.
    __device__ inline void load_k(const Source& s) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) k[i] = *reinterpret_cast<const uintx4*>(s.k + 1024 * i);
        ks = *reinterpret_cast<const uintx4*>(s.ks);
        vs = *reinterpret_cast<const uintx4*>(s.vs);
    }
    __device__ inline void load_v(const Source& s) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) v[i] = *reinterpret_cast<const uintx4*>(s.v + 1024 * i);
        there = s.there;
    }
};

// Lookups run this many products ahead of the matrix instructions.  Two: 64
// contexts of 512-8192 tokens 57.0 -> 54.4 us, three of 66-131k 85.6 -> 80.7,
// more gains nothing; with none fenced off the compiler hoists all and spills.
constexpr int kAhead = 2;

template <int D, int DT, int NT>
struct Wave {
    static constexpr int kDb = D / 16;  // dimension blocks of O
    static constexpr int kKs = D / 32;  // contraction steps of S

    half8 q[NT][kKs];
    floatx4 o[NT][kDb];
    float m[NT], l[NT], qs[NT];  // qs: the power of two that q was divided by
    int lo[NT], hi[NT];  // positions the lane's query row sees
    // v scales up to `limit` (bits of the cache dtype in both halves) times p up
    // to 2^slack give weights up to 2^kTop
    uint32_t limit;
    float slack;
    int inner_lo, inner_hi;  // positions every row of the wave sees

    // The tile's query rows as they are (n may be <= 0), a lane's quarter of
    // a row each.  Separate from init() so that the first codes can be on
    // their way before a row is waited for.
    using Raw = uint32_t[NT][D / 8];
    __device__ static inline void fetch(const AttnArgs& a, const Rows& rw, int h, int lane, Raw& x) {
        const int g = lane >> 4, c = lane & 15;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int w = 0; w < D / 8; ++w) x[t][w] = 0;
            if (t * 16 + c >= rw.n) continue;
            const int r = rw.r0 + t * 16 + c, i = divide(r, a.G, a.G_magic);
            const uint16_t* p = a.q + (int64_t)(rw.tok0 + i) * a.q_token +
                                (int64_t)(h * a.G + r - i * a.G) * a.q_head + g * (D / 4);
            if (a.q_vec) {
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    const uintx4 y = reinterpret_cast<const uintx4*>(p)[w];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[t][4 * w + e] = y[e];
                }
            } else {
#pragma unroll
                for (int w = 0; w < D / 8; ++w) x[t][w] = p[2 * w] | (uint32_t)p[2 * w + 1] << 16;
            }
        }
    }
    __device__ inline void init(const AttnArgs& a, const Rows& rw, const Raw& x, int lane) {
        const int c = lane & 15;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            lo[t] = hi[t] = 0;
            if (t * 16 + c < rw.n)
                bounds(a, rw, divide(rw.r0 + t * 16 + c, a.G, a.G_magic), lo[t], hi[t]);
            // the row's largest magnitude, and the power of two below it
            float big = 0.f;
#pragma unroll
            for (int w = 0; w < D / 8; ++w)
                big = max3(big, fabsf(kv_f32<DT>(x[t][w] & 0xffff)), fabsf(kv_f32<DT>(x[t][w] >> 16)));
            big = max_groups(big);
            int e = (int)(__builtin_bit_cast(uint32_t, big) >> 23 & 0xff);
            e = big == 0.f || e == 255 ? 0 : (e < 1 ? 1 : e) - 127;
            const float f = ldexpf(1.f, -e);
            qs[t] = ldexpf(1.f, e);
#pragma unroll
            for (int s = 0; s < kKs; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t w = x[t][4 * s + j];
                    q[t][s][2 * j] = (_Float16)(kv_f32<DT>(w & 0xffff) * f);
                    q[t][s][2 * j + 1] = (_Float16)(kv_f32<DT>(w >> 16) * f);
                }
            m[t] = kNoMax;
            l[t] = 0.f;
#pragma unroll
            for (int i = 0; i < kDb; ++i) o[t][i] = floatx4{0, 0, 0, 0};
        }
        slack = kMostP;
        limit = 0;  // the first block sets them
        // bounds grow with the row, so the first and last rows tell
        inner_lo = 0;
        inner_hi = 0x7fffffff;
        if (rw.n > 0) {
            int x0, x1;
            bounds(a, rw, divide(rw.r0, a.G, a.G_magic), x0, inner_hi);
            bounds(a, rw, divide(rw.r0 + rw.n - 1, a.G, a.G_magic), inner_lo, x1);
        }
    }

    // One block; `at` is its first position.  The next block's k and v are
    // loaded into the same registers as soon as this one's are done with.
    __device__ inline void step(Block<D>& blk, const Source& next, int at, uint32_t lane4, int g,
                                float qk) {
        // scores
        floatx4 s[2][NT];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int t = 0; t < NT; ++t) s[u][t] = floatx4{0, 0, 0, 0};
        // the lookups of a step ahead of the products of the one before, and no
        // further: unfenced, the compiler hoists them all and runs out of registers
        constexpr int F = kAhead;
        half8 x[F + 1][2];
        auto keys = [&](int c) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int w = u * kKs + c;
                x[c % (F + 1)][u] = lookup<false>(blk.k[w >> 2][w & 3], lane4);
            }
        };
#pragma unroll
        for (int c = 0; c < F && c < kKs; ++c) keys(c);
#pragma unroll
        for (int c = 0; c < kKs; ++c) {
            if (c + F < kKs) keys(c + F);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t) s[u][t] = mfma(x[c % (F + 1)][u], q[t][c], s[u][t]);
        }
        half8 w[NT];
        float ks[8], vs[8], top[NT];
        const uintx4 vw = blk.vs;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            ks[j] = (j & 1 ? high_f32<DT>(blk.ks[j >> 1]) : low_f32<DT>(blk.ks[j >> 1])) * qk;
            vs[j] = j & 1 ? high_f32<DT>(vw[j >> 1]) : low_f32<DT>(vw[j >> 1]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j >> 2][t][j & 3] *= ks[j];
        if (!blk.there || at < inner_lo || at + kKvBlock > inner_hi) {
            // Some row does not see some token.  Scales of tokens that none
            // sees may be anything.
            asm volatile("");  // keeps this a branch: as selects it would run for every block
            const int p0 = at + 8 * g;
            uint32_t seen = 0;  // bit j: some row of this lane sees token j
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint32_t span = blk.there ? hi[t] - lo[t] : 0, from = p0 - lo[t];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool sees = from + j < span;
                    seen |= sees ? 1u << j : 0u;
                    s[j >> 2][t][j & 3] = sees ? s[j >> 2][t][j & 3] : -INFINITY;
                }
            }
            bool nan = false;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                vs[j] = seen >> j & 1 ? vs[j] : 0.f;
                nan |= vs[j] != vs[j];
            }
            if (__any(nan)) {
                // 0 * NaN must not reach the rows that do not see it: the
                // others' results become NaN here, the scale zero
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float hit = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (vs[j] != vs[j] && p0 + j >= lo[t] && p0 + j < hi[t]) hit = 1.f;
                    const float z = max_groups(hit) > 0.f ? __builtin_nanf("") : 0.f;
#pragma unroll
                    for (int i = 0; i < kDb; ++i) o[t][i] += z;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) vs[j] = vs[j] != vs[j] ? 0.f : vs[j];
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float x = max3(s[0][t][0], s[0][t][1], s[0][t][2]);
            x = max3(x, s[0][t][3], s[1][t][0]);
            x = max3(x, s[1][t][1], s[1][t][2]);
            top[t] = max2(x, s[1][t][3]);
        }
        // a weight might pass 2^kTop: by bounds, largest score and largest scale
        const uint32_t bits = max_u16(max_u16(vw[0], vw[1]), max_u16(vw[2], vw[3]));
        blk.load_k(next);
        bool raise = max_u16(bits, limit) != limit;
#pragma unroll
        for (int t = 0; t < NT; ++t) raise |= fmaf(top[t], qs[t], -m[t]) > slack;
        if (__any(raise)) {
            // the bounds of this block's scales, then m by the weights themselves
            float big = vs[0], most[NT];
#pragma unroll
            for (int j = 1; j < 8; ++j) big = fmaxf(big, vs[j]);
            big = max_groups(big);
            const int e = (int)(__builtin_bit_cast(uint32_t, big) >> 23 & 0xff) - 127;
            limit = big > 0.f ? pow2_bits<DT>(e + (int)kRoom) : 0;
            slack = fminf(kTop - kRoom - (float)e, kMostP);
#pragma unroll
            for (int t = 0; t < NT; ++t) most[t] = -INFINITY;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float lv = fmaxf(__builtin_amdgcn_logf(vs[j]), kLeastScale);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    most[t] = fmaxf(most[t], fmaf(s[j >> 2][t][j & 3], qs[t], lv));
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float nm = fmaxf(m[t], max_groups(most[t]) - kFirst);
                const float x = __builtin_amdgcn_exp2f(m[t] - nm);
                m[t] = nm;
                l[t] *= x;
#pragma unroll
                for (int i = 0; i < kDb; ++i) o[t][i] *= x;
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = s[j >> 2][t][j & 3];
                const float p = __builtin_amdgcn_exp2f(fmaf(x, qs[t], -m[t]));
                sum += p;
                w[t][j] = (_Float16)(p * vs[j]);
            }
            l[t] += sum;
        }
        // values
#pragma unroll
        for (int half = 0; half < (D + 127) / 128; ++half) {
            uint32_t col[D < 128 ? 4 : 8];
            if constexpr (D == 64) {
                uint32_t row[4] = {blk.v[0][0], blk.v[0][1], blk.v[0][2], blk.v[0][3]};
                transpose4(row, col);
            } else {
                uint32_t row[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) row[j] = blk.v[2 * half + (j >> 2)][j & 3];
                transpose8(row, col);
            }
            constexpr int n = D < 128 ? 4 : 8;
            half8 x[F + 1];
#pragma unroll
            for (int i = 0; i < F; ++i) x[i] = lookup<true>(col[i], lane4);
#pragma unroll
            for (int i = 0; i < n; ++i) {
                if (i + F < n) x[(i + F) % (F + 1)] = lookup<true>(col[i + F], lane4);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    o[t][8 * half + i] = mfma(x[i % (F + 1)], w[t], o[t][8 * half + i]);
            }
        }
        blk.load_v(next);
    }
};

// Blocks first, first + stride, ... below end (at least one) of a request.
// begin() issues the first loads, ahead of other work; a block's page is
// looked up a step before its codes are loaded.
template <int D>
struct Walk {
    const int32_t* table;  // the request's row
    int h, first, end, stride, page, in;
    Block<D> blk;

    __device__ inline void ahead(const AttnArgs& a, int b) {
        b = b < end ? b : end - 1;
        const int pg = a.bpp == 1 ? b : (int)(((uint64_t)(uint32_t)b * a.bpp_magic) >> 32);
        in = b - pg * (int)a.bpp;
        page = table[pg];
    }
    __device__ inline Source source(const AttnArgs& a, int lane) const {
        Source s;
        s.there = (uint32_t)page < (uint32_t)a.pages;
        const int64_t at = ((int64_t)(s.there ? page : 0) * a.Hkv + h) * 2;
        // uniform offsets, then the lane's
        const int64_t code = (at * a.bpp + in) * (16 * D);
        const int64_t row = at * a.page_size + in * kKvBlock;
        s.k = a.codes + code + lane * 16;
        s.v = a.codes + (code + (int64_t)a.bpp * (16 * D)) + lane * 16;
        s.ks = a.scales + row + 8 * (lane >> 4);
        s.vs = a.scales + (row + a.page_size) + 8 * (lane >> 4);
        return s;
    }
    __device__ inline void begin(const AttnArgs& a, const int32_t* row, int head, int lo, int hi,
                                 int by, int lane) {
        table = row;
        h = head;
        first = lo;
        end = hi;
        stride = by;
        ahead(a, first);
        const Source s = source(a, lane);
        blk.load_k(s);
        blk.load_v(s);
        ahead(a, first + stride);
    }
    template <int DT, int NT>
    __device__ inline void run(const AttnArgs& a, Wave<D, DT, NT>& wv, int lane) {
        const uint32_t lane4 = 4 * (lane & 31);
        const int g = lane >> 4;
        for (int b = first; b < end; b += stride) {
            const Source next = source(a, lane);
            ahead(a, b + 2 * stride);
            wv.step(blk, next, b * kKvBlock, lane4, g, a.qk);
        }
    }
};

// Inclusive scan over the threads of W waves; scratch of W ints.
template <int W>
__device__ inline int group_scan(int x, int* scratch, int& total, int tid) {
    const int lane = tid & 63, wave = tid >> 6;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(x, o);
        if (lane >= o) x += y;
    }
    if (lane == 63) scratch[wave] = x;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const int y = scratch[w];
        if (w < wave) x += y;
        total += y;
    }
    return x;
}

template <int DT>
__device__ inline void store_out(const AttnArgs& a, int64_t tok, int head, int D, int d,
                                 floatx4 x) {
    const uint32_t lo = kv_bits<DT>(x[0]) | kv_bits<DT>(x[1]) << 16;
    const uint32_t hi = kv_bits<DT>(x[2]) | kv_bits<DT>(x[3]) << 16;
    *reinterpret_cast<uint2*>(a.out + (tok * a.Hq + head) * D + d) = make_uint2(lo, hi);
}

// Results of a wave that saw all keys of its rows.
template <int D, int DT, int NT>
__device__ inline void finish(const AttnArgs& a, const Wave<D, DT, NT>& wv, const Rows& rw, int h,
                              int lane) {
    const int g = lane >> 4, c = lane & 15;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float l = wv.l[t];
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (t * 16 + c >= rw.n) continue;
        const int r = rw.r0 + t * 16 + c, i = divide(r, a.G, a.G_magic);
        const int head = h * a.G + r - i * a.G;
        const int64_t tok = rw.tok0 + i;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                floatx4 x;
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = wv.o[t][4 * k + j][e] * inv;
                store_out<DT>(a, tok, head, D, (4 * g + e) * (D / 16) + 4 * k, x);
            }
        if (a.lse && g == 0)
            a.lse[tok * a.Hq + head] = (wv.m[t] + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
    }
}

// ---- rows form: every wave of a workgroup takes other query rows ------------

// Requests that the heavy-first order can sort.
constexpr int kOrderB = 256;

// Grid: row tiles of all requests x kv heads, heads fastest, so that the
// workgroups of a head tend to share an XCD's L2 and the heavy tiles of all
// heads come first.  A workgroup's tile is 4 x 16 NT rows of one request.  Tiles differ in work by as much as the requests'
// lengths, and a workgroup that starts late with a long one holds up the
// end, so they are taken in the order of the keys before their last row, most
// first.  With n_b tiles in request b and o_b tiles' worth of keys before
// them, tile t is at level o_b + t; F(x) = sum_b clamp(o_b + n_b - x, 0, n_b)
// tiles are at level x or above.  Every lane tries another x.  For more than
// kOrderB requests each search would cost as much as it saves: requests in
// order, each from its last tile.
//
// Bound by vector instructions: 336 a block of 48 rows x 128 dimensions
// beside 48 matrix instructions, which two waves a SIMD (251 registers) hardly
// overlap.  Six prompts of 1000-4096 tokens, 32 / 8 heads of 128: 482 us, 763
// TFLOP/s.  In an earlier build, tiles in order of requests took 652 us; 32 rows
// a wave 736 us; 64 rows spill inside the loop, 1150 us.
template <int D, int DT, int NT>
__global__ __launch_bounds__(kAttnThreads, 2) void k_kv4_attn_rows(AttnArgs a) {
    extern __shared__ uint32_t tab[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    constexpr int rows = 16 * NT * kAttnWaves;
    const int want = blockIdx.x / (uint32_t)a.Hkv, h = blockIdx.x - want * a.Hkv;
    int b = 0, tile = 0;
    if (a.B <= kOrderB) {
        int2* req = reinterpret_cast<int2*>(tab);  // (o_b, n_b)
        int* most = reinterpret_cast<int*>(req + kOrderB);
        if (tid == 0) most[0] = most[1] = 0;
        __syncthreads();
        if (tid < a.B) {
            Rows rw;
            request_lens(a, tid, rw);
            const int n = (rw.qlen * a.G + rows - 1) / rows;
            const int before = a.causal ? rw.seq - rw.qlen : rw.seq;
            const int64_t level = before < 0 ? 0 : (int64_t)before * a.G / rows;
            const int o = level > 1 << 29 ? 1 << 29 : (int)level;
            req[tid] = make_int2(o, n);
            atomicMax(&most[0], o + n);
            atomicAdd(&most[1], n);
        }
        __syncthreads();
        if (want >= most[1]) return;
        int lo = 0, len = most[0];  // F(lo) > want, F(lo + len) <= want
        while (len > 1) {
            const int step = (len + 63) / 64, x = lo + lane * step;
            int f = 0;
            for (int i = 0; i < a.B; ++i) {
                const int2 r = req[i];
                const int c = r.x + r.y - x;
                f += c < 0 ? 0 : c > r.y ? r.y : c;
            }
            const int k = __popcll(__ballot(lane * step < len && f > want)) - 1;
            lo += k * step;
            len = len - k * step < step ? len - k * step : step;
        }
        int f = 0;  // tiles above the level
        for (int i = lane; i < a.B; i += 64) {
            const int2 r = req[i];
            const int c = r.x + r.y - lo - 1;
            f += c < 0 ? 0 : c > r.y ? r.y : c;
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) f += __shfl_xor(f, o);
        int rank = want - f;  // within the level
        for (int i0 = 0; i0 < a.B; i0 += 64) {
            const int2 r = i0 + lane < a.B ? req[i0 + lane] : make_int2(0, 0);
            uint64_t m = __ballot(lo >= r.x && lo < r.x + r.y);
            const int k = __popcll(m);
            if (rank < k) {
                for (; rank > 0; --rank) m &= m - 1;
                b = i0 + __builtin_ctzll(m);
                tile = lo - req[b].x;
                break;
            }
            rank -= k;
        }
    } else {
        int* scratch = reinterpret_cast<int*>(tab);
        int* found = scratch + kAttnWaves;
        const int per = (a.B + kAttnThreads - 1) / kAttnThreads, b0 = tid * per;
        int mine = 0, total;
        Rows rw;
        for (int i = b0; i < b0 + per && i < a.B; ++i) {
            request_lens(a, i, rw);
            mine += (rw.qlen * a.G + rows - 1) / rows;
        }
        int before = group_scan<kAttnWaves>(mine, scratch, total, tid) - mine;
        if (want >= total) return;
        if (want >= before && want < before + mine) {
            for (int i = b0;; ++i) {
                request_lens(a, i, rw);
                const int n = (rw.qlen * a.G + rows - 1) / rows;
                if (want < before + n) {
                    found[0] = i;
                    found[1] = n - 1 - (want - before);
                    break;
                }
                before += n;
            }
        }
        __syncthreads();
        b = found[0];
        tile = found[1];
    }
    b = __builtin_amdgcn_readfirstlane(b);
    tile = __builtin_amdgcn_readfirstlane(tile);
    __syncthreads();
    Rows rw;
    request_lens(a, b, rw);
    const Span sp = tile_rows(a, rw, tile * rows + wave * 16 * NT, 16 * NT);
    typename Wave<D, DT, NT>::Raw raw;
    Wave<D, DT, NT>::fetch(a, rw, h, lane, raw);
    Walk<D> wk;
    if (sp.hi > sp.lo) wk.begin(a, a.table + b * a.max_pages, h, sp.lo, sp.hi, 1, lane);
    build_table(tab, a.codebook, a.Hkv, h, tid, kAttnThreads);
    Wave<D, DT, NT> wv;
    wv.init(a, rw, raw, lane);
    __syncthreads();
    if (sp.hi > sp.lo) wk.run(a, wv, lane);
    finish<D, DT, NT>(a, wv, rw, h, lane);
}

// ---- few query rows: row tiles of requests ----------------------------------------

// Row tile rt of request b, and its visible blocks.
template <int NT>
__device__ inline Span split_span(const AttnArgs& a, int b, int rt, Rows& rw) {
    request_lens(a, b, rw);
    return tile_rows(a, rw, rt * 16 * NT, 16 * NT);
}

// ---- group form: a few waves a (request, row tile, kv head) -----------------------

// Adds up the S waves of a group and writes their rows.  ml: [16 NT][W].
template <int S, int W, int D, int DT, int NT>
__device__ inline void group_merge(const AttnArgs& a, const Wave<D, DT, NT>& wv, const Rows& rw,
                                   uint32_t* tab, float2* ml, int h, int wave, int lane) {
    const int sub = wave & (S - 1), wave0 = wave - sub, c = lane & 15;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float l = wv.l[t];
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (lane < 16) ml[(t * 16 + c) * W + wave] = make_float2(wv.m[t], l);
    }
    __syncthreads();
    floatx4* buf = reinterpret_cast<floatx4*>(tab);  // [W][D / 16][64]: accumulators of a wave
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float top = kNoMax;
#pragma unroll
        for (int w = 0; w < S; ++w) top = fmaxf(top, ml[(t * 16 + c) * W + wave0 + w].x);
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
        for (int i = sub * 64 + lane; i < 4 * D; i += 64 * S) {
            const int p = i >> 6, e = p / (D / 64), k = p % (D / 64), row = t * 16 + (i & 15);
            if (row >= rw.n) continue;
            floatx4 x = buf[wave0 * 4 * D + i];
#pragma unroll
            for (int w = 1; w < S; ++w) x += buf[(wave0 + w) * 4 * D + i];
            float most = kNoMax, sum = 0.f;
#pragma unroll
            for (int w = 0; w < S; ++w) most = fmaxf(most, ml[row * W + wave0 + w].x);
#pragma unroll
            for (int w = 0; w < S; ++w) {
                const float2 y = ml[row * W + wave0 + w];
                sum += y.y * __builtin_amdgcn_exp2f(y.x - most);
            }
            const int r = rw.r0 + row, q = divide(r, a.G, a.G_magic), head = h * a.G + r - q * a.G;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const int d = (4 * ((i >> 4) & 3) + e) * (D / 16) + 4 * k;
            store_out<DT>(a, rw.tok0 + q, head, D, d, x * inv);
            if (a.lse && d == 0)
                a.lse[(int64_t)(rw.tok0 + q) * a.Hq + head] =
                    (most + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
        }
        if (t + 1 < NT) __syncthreads();
    }
}

// Grid (requests / groups, row tiles x kv heads).  A workgroup's W waves are
// groups of a.group; the waves of a group take every a.group-th block of their
// request and their sums meet in LDS, over the table, which nobody needs by
// then.  Bound by the chain lengths -> page -> codes -> merge and the blocks of
// the longest request: one context of 257 tokens 8.1 us (groups of 8), 256
// contexts of 16-600, 64 / 8 heads of 128, 27 us (of 1).
template <int D, int DT, int NT>
__global__ __launch_bounds__((64 * kSplitWaves<D, NT>), (kSplitWaves<D, NT> / 2))
void k_kv4_attn_group(AttnArgs a) {
    constexpr int W = kSplitWaves<D, NT>, kThreads = 64 * W;
    extern __shared__ uint32_t tab[];
    float2* ml = reinterpret_cast<float2*>(tab + kTabBytes / 4);  // [16 NT][W]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int S = a.group, sub = wave & (S - 1), wave0 = wave - sub;  // of the group
    const int b = (blockIdx.x * W + wave0) / (uint32_t)S;
    const int h = blockIdx.y / a.row_tiles, rt = blockIdx.y - h * a.row_tiles;
    Rows rw{};
    Span sp = {0, 0};
    if (b < a.B) sp = split_span<NT>(a, b, rt, rw);
    const bool some = sp.lo + sub < sp.hi;
    typename Wave<D, DT, NT>::Raw raw;
    Wave<D, DT, NT>::fetch(a, rw, h, lane, raw);
    Walk<D> wk;
    if (some) wk.begin(a, a.table + b * a.max_pages, h, sp.lo + sub, sp.hi, S, lane);
    build_table(tab, a.codebook, a.Hkv, h, tid, kThreads);
    Wave<D, DT, NT> wv;
    wv.init(a, rw, raw, lane);
    __syncthreads();
    if (some) wk.run(a, wv, lane);
    if (S == 1) {
        finish<D, DT, NT>(a, wv, rw, h, lane);
        return;
    }
    if (S == 2) group_merge<2, W, D, DT, NT>(a, wv, rw, tab, ml, h, wave, lane);
    else if (S == 4) group_merge<4, W, D, DT, NT>(a, wv, rw, tab, ml, h, wave, lane);
    else if constexpr (W == 8) group_merge<8, W, D, DT, NT>(a, wv, rw, tab, ml, h, wave, lane);
}

// ---- split form: shares of the keys, a wave each ----------------------------------

// Blocks a wave takes of `total` (< 2^31): an equal share; more, up to `least`,
// where an eighth of the waves is enough for that.
__device__ inline int split_share(uint32_t total, uint32_t waves, int least) {
    const int per = (int)((total + waves - 1) / waves);
    const int eighth = (int)((total + waves / 8) / (waves / 8 + 1));
    const int more = eighth < least ? eighth : least;
    const int share = per > more ? per : more;
    return share < 2 ? 2 : share;
}

// Sums of a share of a request, for the join.
template <int D, int DT, int NT>
__device__ inline void store_part(const AttnArgs& a, const Wave<D, DT, NT>& wv, const Rows& rw,
                                  int64_t part, int lane) {
    const int g = lane >> 4, c = lane & 15;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float l = wv.l[t];
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (t * 16 + c >= rw.n) continue;
        const int64_t row = part * a.part_rows + t * 16 + c;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                floatx4 x;
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = wv.o[t][4 * k + j][e];
                *reinterpret_cast<floatx4*>(a.part_o + row * D + (4 * g + e) * (D / 16) + 4 * k) = x;
            }
        if (g == 0) *reinterpret_cast<float2*>(a.part_ml + row * 2) = make_float2(wv.m[t], l);
    }
}

// Grid (splits, row tiles x kv heads).  The blocks of a (row tile, head) over
// all requests form one line that is cut into equal shares, whatever the
// lengths, one a wave.  A wave walks its share request by request; a request
// that lies whole in it is finished there, else its sums go to the workspace
// and k_kv4_attn_join adds the shares of a request in order.  Waves meet
// nowhere after the table is built.
//
// Three contexts of 66-131k tokens, 32 / 8 heads of 128: 78 us with the join,
// 4.2 TB/s of codes and scales, near what a copy reaches.  64 contexts of
// 512-8192: 53 us, 3.3 TB/s; 8 us of it pass before a wave has its first codes
// and 6 us in the join.  One share a wave and no more (two rounds: 70 us).
template <int D, int DT, int NT>
__global__ __launch_bounds__((64 * kSplitWaves<D, NT>), (kSplitWaves<D, NT> / 2))
void k_kv4_attn_split(AttnArgs a) {
    constexpr int W = kSplitWaves<D, NT>, kThreads = 64 * W;
    extern __shared__ uint32_t tab[];
    int* scratch = reinterpret_cast<int*>(tab + kTabBytes / 4);
    struct Start {  // where a share begins: a request, how many of its blocks lie before
        int b, skip, tok0, qlen, seq;
    };
    Start* start = reinterpret_cast<Start*>(scratch + W);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = blockIdx.y / a.row_tiles, rt = blockIdx.y - h * a.row_tiles;
    const int per = (a.B + kThreads - 1) / kThreads, b0 = tid * per;
    Rows rw;
    int mine = 0, total;
    Span sp = {0, 0};
    for (int b = b0; b < b0 + per && b < a.B; ++b) {
        sp = split_span<NT>(a, b, rt, rw);
        mine += sp.hi - sp.lo;
    }
    build_table(tab, a.codebook, a.Hkv, h, tid, kThreads);
    int at = group_scan<W>(mine, scratch, total, tid) - mine;
    const int share = split_share(total, a.splits * W, a.least);
    const int first_wave = blockIdx.x * W;
    // Where the shares of this workgroup begin, and what the join needs.
    const bool tell = blockIdx.x == 0 && h == 0;
    const int64_t begin = (int64_t)first_wave * share, stop = begin + (int64_t)W * share;
    if (tell || (at < stop && at + mine > begin)) {
        int* prefix = a.prefix + (int64_t)rt * (a.B + 1);
        for (int b = b0; b < b0 + per && b < a.B; ++b) {
            if (per > 1) sp = split_span<NT>(a, b, rt, rw);
            const int n = sp.hi - sp.lo;
            if (tell) prefix[b] = at;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const int64_t from = begin + w * share;
                if (from >= at && from < at + n)
                    start[w] = {b, (int)(from - at), rw.tok0, rw.qlen, rw.seq};
            }
            at += n;
        }
        if (tell && tid == 0) a.prefix[(int64_t)rt * (a.B + 1) + a.B] = total;
    }
    if (begin >= total) return;
    __syncthreads();

    const int64_t over = total - (begin + wave * share);  // blocks from the wave's share on
    int left = over > share ? share : (int)over;          // of the share
    if (left <= 0) return;
    const int64_t part = ((int64_t)blockIdx.y * a.splits * W + first_wave + wave) * 2;
    int b = __builtin_amdgcn_readfirstlane(start[wave].b);
    int skip = __builtin_amdgcn_readfirstlane(start[wave].skip);
    rw.tok0 = __builtin_amdgcn_readfirstlane(start[wave].tok0);
    rw.qlen = __builtin_amdgcn_readfirstlane(start[wave].qlen);
    rw.seq = __builtin_amdgcn_readfirstlane(start[wave].seq);
    for (int place = 0;;) {
        sp = tile_rows(a, rw, rt * 16 * NT, 16 * NT);
        const int all = sp.hi - sp.lo;
        if (all > 0) {
            const int take = all - skip < left ? all - skip : left;
            typename Wave<D, DT, NT>::Raw raw;
            Wave<D, DT, NT>::fetch(a, rw, h, lane, raw);
            Walk<D> wk;
            wk.begin(a, a.table + b * a.max_pages, h, sp.lo + skip, sp.lo + skip + take, 1, lane);
            Wave<D, DT, NT> wv;
            wv.init(a, rw, raw, lane);
            wk.run(a, wv, lane);
            if (take == all) finish<D, DT, NT>(a, wv, rw, h, lane);
            else store_part<D, DT, NT>(a, wv, rw, part + place, lane);
            left -= take;
            if (left <= 0) return;
            place = 1;  // the share's first request has place 0, its last place 1
            skip = 0;
        }
        request_lens(a, ++b, rw);
    }
}

// Adds the shares of requests that lie in several, in their order, and writes
// zeros for rows that see nothing.  Grid (B, row tiles x kv heads, z): a
// workgroup takes every z-th row, join_rows of them at once; the threads of a
// row are D/4 wide, four dimensions each, and take every n-th share.
template <int D, int DT, int NT>
__global__ __launch_bounds__(kAttnThreads) void k_kv4_attn_join(AttnArgs a) {
    constexpr int kGroups = kAttnThreads / (D / 4);
    __shared__ floatx4 so[kAttnThreads];
    __shared__ float sm[kGroups], sl[kGroups];
    const int b = blockIdx.x;
    const int h = blockIdx.y / a.row_tiles, rt = blockIdx.y - h * a.row_tiles;
    const int* prefix = a.prefix + (int64_t)rt * (a.B + 1);
    const int lo = prefix[b], hi = prefix[b + 1], total = prefix[a.B];
    Rows rw;
    split_span<NT>(a, b, rt, rw);
    const int waves = a.splits * kSplitWaves<D, NT>, share = split_share(total, waves, a.least);
    const int w0 = lo / share, w1 = hi > lo ? (hi - 1) / share : w0;
    if (hi > lo && w0 == w1) return;
    const int tid = threadIdx.x, grp = tid / (D / 4), d = 4 * (tid % (D / 4));
    const int n = kGroups / a.join_rows, sub = grp % n;  // threads of a row, which of them
    for (int r0 = 0; r0 * (int)gridDim.z < rw.n; r0 += a.join_rows) {
        const int row = (r0 + grp / n) * gridDim.z + blockIdx.z;
        float top = kNoMax, sum = 0.f;
        floatx4 o = {0, 0, 0, 0};
        if (hi > lo && row < rw.n) {
            constexpr int kBatch = 4;  // shares loaded at a time
            for (int w = w0 + sub; w <= w1; w += kBatch * n) {
                float2 ml[kBatch];
                floatx4 y[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int x = w + i * n <= w1 ? w + i * n : w;
                    const int64_t part = (((int64_t)blockIdx.y * waves + x) * 2 +
                                          (x == w0 && lo != x * share ? 1 : 0)) * a.part_rows + row;
                    ml[i] = *reinterpret_cast<const float2*>(a.part_ml + part * 2);
                    y[i] = *reinterpret_cast<const floatx4*>(a.part_o + part * D + d);
                }
                float nm = top;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) nm = fmaxf(nm, ml[i].x);
                float f = __builtin_amdgcn_exp2f(top - nm);
                o *= f;
                sum *= f;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    f = w + i * n <= w1 ? __builtin_amdgcn_exp2f(ml[i].x - nm) : 0.f;
                    o += y[i] * f;
                    sum += ml[i].y * f;
                }
                top = nm;
            }
        }
        if (n > 1) {
            so[tid] = o;
            if (d == 0) {
                sm[grp] = top;
                sl[grp] = sum;
            }
            __syncthreads();
            if (sub == 0) {
                float all = top;
                for (int i = 1; i < n; ++i) all = fmaxf(all, sm[grp + i]);
                float f = __builtin_amdgcn_exp2f(top - all);
                sum *= f;
                o *= f;
                for (int i = 1; i < n; ++i) {
                    f = __builtin_amdgcn_exp2f(sm[grp + i] - all);
                    sum += sl[grp + i] * f;
                    o += so[tid + i * (D / 4)] * f;
                }
                top = all;
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

// ---- launches ------------------------------------------------------------------

template <int D, int DT, int NT>
hipError_t attn_rows(const AttnArgs& a, hipStream_t s) {
    static LdsAttr rec;
    auto kern = k_kv4_attn_rows<D, DT, NT>;
    hipError_t e = ensure_lds(rec, reinterpret_cast<const void*>(kern), kTabBytes);
    if (e != hipSuccess) return e;
    constexpr int rows = 16 * NT * kAttnWaves;
    const int64_t tiles = (a.T * a.G + rows - 1) / rows + a.B;
    kern<<<dim3((unsigned)(tiles * a.Hkv)), dim3(kAttnThreads), kTabBytes, s>>>(a);
    return hipGetLastError();
}

template <int D, int DT, int NT>
hipError_t attn_group(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
    static LdsAttr rec;
    constexpr int W = kSplitWaves<D, NT>, lds = kTabBytes + 16 * NT * W * 8;
    auto kern = k_kv4_attn_group<D, DT, NT>;
    hipError_t e = ensure_lds(rec, reinterpret_cast<const void*>(kern), lds);
    if (e != hipSuccess) return e;
    const int64_t each = W / p.group;  // requests a workgroup
    kern<<<dim3((unsigned)((a.B + each - 1) / each), (unsigned)(a.Hkv * p.row_tiles)), dim3(64 * W),
           lds, s>>>(a);
    return hipGetLastError();
}

template <int D, int DT, int NT>
hipError_t attn_split(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
    if (p.group) return attn_group<D, DT, NT>(a, p, s);
    static LdsAttr rec;
    auto kern = k_kv4_attn_split<D, DT, NT>;
    hipError_t e = ensure_lds(rec, reinterpret_cast<const void*>(kern), kSplitLds);
    if (e != hipSuccess) return e;
    const unsigned y = (unsigned)(a.Hkv * p.row_tiles);
    kern<<<dim3((unsigned)p.splits, y), dim3(64 * kSplitWaves<D, NT>), kSplitLds, s>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_kv4_attn_join<D, DT, NT>
        <<<dim3((unsigned)a.B, y, (unsigned)p.join_z), dim3(kAttnThreads), 0, s>>>(a);
    return hipGetLastError();
}

template <int D, int DT>
hipError_t attn_cols(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
    if (!p.split) return attn_rows<D, DT, kRowCols<D>>(a, s);
    if constexpr (kTileCols<D> > 1) {
        if (p.col_blocks == 2) return attn_split<D, DT, 2>(a, p, s);
        if (p.col_blocks == 3) return attn_split<D, DT, 3>(a, p, s);
    }
    return attn_split<D, DT, 1>(a, p, s);
}

template <int D>
hipError_t attn_d(const AttnArgs& a, const AttnPlan& p, int dtype, hipStream_t s) {
    return dtype == FK_BF16 ? attn_cols<D, FK_BF16>(a, p, s) : attn_cols<D, FK_F16>(a, p, s);
}

}  // namespace
}  // namespace fk
