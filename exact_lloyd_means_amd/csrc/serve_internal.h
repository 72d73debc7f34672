// serve_internal.h -- declarations shared by the translation units of the
// operators around a serving step (include/fk_serve.h).
#pragma once

#include "../../include/fk_serve.h"
#include "kv4_internal.h"

namespace fk {

// ---- rotary positions ---------------------------------------------------------
struct RopeSet {
    const void* x;
    void* y;
    int64_t x_token, x_head, y_token, y_head;
};
struct RopeArgs {
    RopeSet set[2];
    int32_t heads[2];
    int64_t T;
    int32_t D, R;
    int32_t units, turn_units;  // accesses of a row; those that are rotated
    const int32_t* pos;
    const uint64_t* turns;
    float factor, sin_factor;   // the latter negative for the inverse
};
hipError_t launch_rope(const RopeArgs& a, int dtype, bool inter, hipStream_t s);

// ---- verification of drafts -----------------------------------------------------
struct VerifyArgs {
    int64_t B, T, V;
    const int32_t *cu, *tokens, *seq;
    const void *p, *q;
    int64_t p_row, q_row;
    const float *u, *pick;
    int32_t *accepted, *emitted, *keep;
    int32_t pieces, len;  // of a row; elements of one
    uint64_t* sums;       // sampling: [B][pieces][2]; greedy: [T][pieces]
    int32_t* kept;        // sampling: [B] 2 drafts kept, + 1 unless the next is no token
};
// Pieces a row of V is cut into where `rows` of them are read.
int verify_pieces(int64_t rows, int64_t V, bool greedy);
// Pieces of all rows together, at most, of up to so many rows of up to V.
int64_t verify_most_pieces(int64_t rows, int64_t V, bool greedy);
hipError_t launch_verify(const VerifyArgs& a, int dtype, hipStream_t s);

// ---- pages ------------------------------------------------------------------------
struct ForkArgs {
    int64_t R, M, N;  // rows, max_pages, pages
    int32_t n, P;
    const int32_t *rows, *sources, *keep;
    int32_t *table, *lens, *shares, *free_pages, *free_count, *copies, *seq;
    int32_t* info;   // [n][8]
    int32_t* fresh;  // [n][M] entries of the sources
    int32_t* have;   // [2] pages of the list before the copies, pages taken
    int32_t *count, *tail, *next;  // [N] change of the holders, first row that
                                   // goes on in the page, new shares
    uint64_t* first;               // [N] first entry that gives the page up
    // of many pairs, else null:
    int32_t* named;  // [R][2] first pair that names a row, least of its lengths
    int32_t* upto;   // [n][2] pages given up and copies of the pairs before
};
constexpr int kForkMany = 1024;  // pairs from which on these are made
hipError_t launch_kv_fork(const ForkArgs& a, hipStream_t s);

struct CompactArgs {
    int64_t R, M, N, n_moves;
    int32_t P;
    const int32_t *table, *lens, *shares, *free_pages, *free_count;
    int32_t *new_table, *new_shares, *new_free, *free_left, *moves;
    uint32_t* bits;   // [words] free pages
    int32_t* before;  // [words + 1] free pages before each word
};
hipError_t launch_kv_compact(const CompactArgs& a, hipStream_t s);

struct CopyArgs {
    uint8_t* codes;
    uint16_t* scales;
    const int32_t* copies;
    int64_t pages;
    int32_t n, P, H, D;
};
hipError_t launch_kv4_copy(const CopyArgs& a, hipStream_t s);

// ---- attention of shared prefixes -------------------------------------------------
constexpr int kSharedGroups = 256;   // most groups that the plan holds in LDS
constexpr int kSharedUnit = 6;       // what a unit of a share costs beside its blocks, in blocks

struct SharedArgs {       // beside AttnArgs, whose part_o and part_ml are the segments' sums
                          // [heads][wgs][16 NA rows]
    const int32_t *cu_groups, *prefix;
    int32_t groups, wgs;  // wgs: workgroups of a head
    int32_t* head;        // [3] lengths of shares, and how many have the first
    int4* unit;           // [units][3] for the join: first token, tokens, length, group or -1; place
                          // in the line, own blocks; first row in the group's tiles, first
                          // segment, segments of a tile
    float *own_o, *own_ml;  // sums of units and shares: [heads][units + 8 wgs][part_rows]
};
struct SharedPlan {
    bool use;             // else as if nothing were shared
    int col_blocks, group_cols;  // blocks of 16 rows of a request's tile, a group's
    int row_tiles, rows, least, join_z, join_rows, wgs;
    size_t head, unit, part_o, part_ml, own_o, own_ml, total;
};
hipError_t launch_kv4_shared_d64(const AttnArgs& a, const SharedArgs& s, const SharedPlan& p, int dtype, hipStream_t st);
hipError_t launch_kv4_shared_d128(const AttnArgs& a, const SharedArgs& s, const SharedPlan& p, int dtype, hipStream_t st);
hipError_t launch_kv4_shared_d256(const AttnArgs& a, const SharedArgs& s, const SharedPlan& p, int dtype, hipStream_t st);

}  // namespace fk
