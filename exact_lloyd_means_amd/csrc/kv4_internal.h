// kv4_internal.h -- declarations shared by the translation units of the
// 4-bit paged cache (include/fk_kv4.h).
#pragma once

#include "../../include/fk_kv4.h"
#include "fk_internal.h"

namespace fk {

constexpr int kKvBlock = 32;  // tokens of a code block

// A 16-bit value of the cache dtype as fp32, and back (nearest even).
template <int DT>
__device__ inline float kv_f32(uint32_t bits) {
    if constexpr (DT == FK_BF16)
        return __builtin_bit_cast(float, bits << 16);
    else
        return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}
template <int DT>
__device__ inline uint32_t kv_bits(float x) {
    if constexpr (DT == FK_BF16)
        return __builtin_bit_cast(uint16_t, (__bf16)x);
    else
        return __builtin_bit_cast(uint16_t, (_Float16)x);
}

typedef unsigned short ushortx2 __attribute__((ext_vector_type(2)));
__device__ inline uint32_t max_u16(uint32_t x, uint32_t y) {  // of both halves
    return __builtin_bit_cast(uint32_t,
                              __builtin_elementwise_max(__builtin_bit_cast(ushortx2, x),
                                                        __builtin_bit_cast(ushortx2, y)));
}
struct PlanArgs {
    int64_t B, max_pages, free_cap, slot_cap;
    int32_t page_size;
    const int32_t *ctx, *fresh, *free_pages, *free_count;
    int32_t *table, *seq, *cu, *slots, *pos, *free_left, *status;
    int32_t* kept;  // [B] or null
    int32_t* ws;  // [B] first needed page of each request, then the list's length
};
hipError_t launch_kv_plan(const PlanArgs& a, hipStream_t s);

struct RowArgs {
    uint8_t* codes;
    uint16_t* scales;
    const uint16_t* codebook;
    const int32_t* slots;
    const uint16_t *k, *v;   // write: inputs
    uint16_t *ko, *vo;       // read: outputs
    int64_t k_token, k_head, v_token, v_head;
    int64_t T, slots_total;  // pages * page_size
    int32_t page_size, H;
    uint32_t bpp, bpp_magic;  // blocks per page; ceil(2^32 / bpp)
};
hipError_t launch_kv4_write(const RowArgs& a, int D, int dtype, bool vec, hipStream_t s);
hipError_t launch_kv4_read(const RowArgs& a, int D, int dtype, hipStream_t s);

struct AttnArgs {
    const uint8_t* codes;
    const uint16_t* scales;
    const uint16_t* codebook;
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    const int32_t *cu, *seq, *table;
    int64_t q_token, q_head, T, max_pages;
    int64_t pages;
    int32_t B, Hq, Hkv, G, page_size, causal, window;
    int32_t max_q;        // most query tokens of a request; more are left out
    int32_t q_vec;        // q rows can be read 16 bytes at a time
    uint32_t bpp, bpp_magic;  // blocks per page; ceil(2^32 / bpp)
    uint32_t G_magic;         // ceil(2^32 / G)
    int32_t cap;              // positions that the table has room for
    int32_t least;            // split form: least blocks of a share
    float qk;             // scale * log2 e
    int32_t group;        // group form: waves of a request
    int32_t row_tiles;    // split form: tiles of query rows of one request
    int32_t splits;       // split form: workgroups per (kv head, row tile)
    int32_t part_rows;    // split form: most rows of a tile
    int32_t join_rows;    // join: rows of a workgroup at a time
    float* part_o;        // split form: [Hkv * row_tiles][waves][2][part_rows][D]
    float* part_ml;       //             [Hkv * row_tiles][waves][2][part_rows][2]
    int32_t* prefix;      //             [row_tiles][B + 1] blocks before each request
};

// Most blocks of 16 query rows of a wave, by head dimension, in the rows form
// and in the others: what the loop over blocks holds in 256 registers.  Around
// that loop the split form of 128 dimensions keeps 21 registers in scratch for
// three blocks of rows and 2 for one; no form touches scratch inside it.
template <int D>
constexpr int kRowCols = D == 64 ? 4 : D == 128 ? 3 : 1;
template <int D>
constexpr int kTileCols = D <= 128 ? 3 : 1;
inline int row_cols(int D) { return D == 64 ? kRowCols<64> : D == 128 ? kRowCols<128> : kRowCols<256>; }
inline int tile_cols(int D) { return D <= 128 ? kTileCols<128> : kTileCols<256>; }

// Waves of a workgroup of the forms for few rows: with one column block of at
// most 128 dimensions four waves fit a SIMD (128 registers), else two.
constexpr int split_waves(int D, int cols) { return cols == 1 && D <= 128 ? 8 : 4; }
template <int D, int NT>
constexpr int kSplitWaves = split_waves(D, NT);

// Query rows of a tile (16 per matrix column block) and the form a call runs.
struct AttnPlan {
    int col_blocks;   // split form: blocks of 16 query rows per wave
    bool split;       // row tiles of requests, else rows
    int group;        // group form: waves of a request, else 0: shares
    int row_tiles, splits;
    int rows;         // split form: most rows of a tile
    int least;        // split form: least blocks of a share
    int join_z, join_rows;  // join: workgroups of a tile, rows of one at a time
    size_t part_o, part_ml, prefix, total;  // workspace: offsets and size
};
AttnPlan plan_attention(int64_t B, int64_t T, int Hq, int Hkv, int D, int max_q,
                        int64_t max_blocks);

// Checks of a cache's shape and addresses.
fk_status kv4_check_cache(const fk_kv4_cache* c);
// Checks of the attention's arguments, and what they say (all but the plan).
fk_status kv4_attn_args(const fk_kv4_cache* c, const fk_kv4_attn* p, AttnArgs& a);

hipError_t launch_kv4_attn_d64(const AttnArgs& a, const AttnPlan& p, int dtype, hipStream_t s);
hipError_t launch_kv4_attn_d128(const AttnArgs& a, const AttnPlan& p, int dtype, hipStream_t s);
hipError_t launch_kv4_attn_d256(const AttnArgs& a, const AttnPlan& p, int dtype, hipStream_t s);

}  // namespace fk
