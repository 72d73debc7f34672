/*
 * fk_serve.h -- what a serving step on the paged 4-bit cache of fk_kv4.h needs
 * around it, for AMD Instinct MI355X (gfx950): rotary positions, attention of
 * requests that share a prefix, verification of drafted tokens, and the pages
 * of a cache forked, returned, copied and compacted.
 *
 * Conventions are those of fk.h and fk_kv4.h (streams, workspaces, errors,
 * nothing allocated or kept).  int32 and fp32 arrays need 4-byte alignment,
 * rows of values that of their type, workspaces 16 bytes.  Results do not
 * depend on timing.
 */
#ifndef FK_SERVE_H
#define FK_SERVE_H

#include "fk_kv4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows of heads: element (t, h, i) of x is at x[t * x_token + h * x_head + i],
 * of y likewise; strides in elements, >= 0.  Rows of x may overlap (a head that
 * is broadcast), those of y may not: strides that make rows of a set share an
 * element are refused, and so are two sets with one y. */
typedef struct fk_rope_rows {
    const void* x;
    void* y;               /* may be x with the same strides; else no overlap */
    int64_t x_token, x_head, y_token, y_head;
    int32_t heads;
    int32_t reserved;      /* 0 */
} fk_rope_rows;

typedef struct fk_rope_args {
    int64_t T;             /* tokens */
    int32_t head_dim;      /* D, even, at most 1024 */
    int32_t rot_dim;       /* R, even, 2 .. D: what is rotated */
    int32_t dtype;         /* FK_F32, FK_F16 or FK_BF16 */
    int32_t interleaved;   /* pair i is (2i, 2i + 1); 0: (i, i + R/2) */
    int32_t inverse;       /* rotate by the negative angle: the gradient */
    float factor;          /* of the rotated part, finite */
    const int32_t* positions; /* [T] */
    const uint64_t* turns; /* [R/2] turns a position advances pair i, in units
                              of 2^-64 turn (w_i / 2 pi 2^64, modulo 2^64);
                              8-byte alignment */
} fk_rope_args;

/*
 * fk_rope -- rotary positions of queries and keys in one pass.  Pair i of a
 * token at position p, as a complex number z, becomes factor z e^(2 pi j p
 * turns_i); elements from R on are copied, and so are whole rows of tokens at
 * negative positions.  The angle is a product of integers and exact for every
 * position; sine and cosine, products and sums are fp32, rounded once to the
 * type.  n is 1 or 2 sets of rows (queries; keys) that share the positions.
 * With inverse it is the transposed map, so the gradient with respect to x is
 * that of y rotated back.  T <= 2^24, heads <= 2^16.
 */
fk_status fk_rope(const fk_rope_args* a, int32_t n, const fk_rope_rows* rows, void* stream);

typedef struct fk_verify_args {
    int64_t B;             /* requests, <= 2^20 */
    int64_t T;             /* rows of all requests, <= 2^24 */
    int64_t V;             /* tokens of the vocabulary, <= 2^20 */
    const int32_t* cu;     /* [B+1] first row of each request */
    const int32_t* tokens; /* [T] the step's input tokens; those of a request
                              after its first are drafts */
    const void* target;    /* (T, V): row r is the target's distribution of
                              the token after row r */
    const void* draft;     /* (T, V): what tokens[r + 1] was drawn from; NULL:
                              drafts are certain.  A request's last row is
                              not read */
    int64_t target_row, draft_row; /* row strides in elements, >= 0 */
    int32_t dtype;         /* of both */
    int32_t reserved;      /* 0 */
    const float* accept;   /* [T] uniform numbers in [0, 1): accept[r] decides
                              tokens[r + 1]; NULL: greedy */
    const float* pick;     /* [B] uniform numbers in [0, 1) (with accept) */
    const int32_t* seq_lens; /* [B] tokens of each request, the step's among
                              them; or NULL */
    int32_t* accepted;     /* [B] drafts kept */
    int32_t* emitted;      /* [T] from cu[b] on: the drafts kept, one token
                              more, then -1; not tokens itself */
    int32_t* keep;         /* [B] seq - drafts not kept; or NULL */
} fk_verify_args;

/* Bytes of workspace for fk_verify of up to so many requests, rows and tokens of
 * the vocabulary (0 when the sizes are invalid). */
size_t fk_verify_workspace_bytes(int64_t B, int64_t T, int64_t V);

/*
 * fk_verify -- which drafted tokens the target keeps, and the token after
 * them.  With p and q rows of target and draft in fp32, u = accept and d =
 * tokens[r + 1]: drafts are kept up to the first with not u q(d) < p(d) (q(d)
 * = 1 without draft; compared exactly), so each token emitted is distributed
 * as p says.  The token after them is i with probability w_i / sum w, where w
 * = max(0, p - q) of the row of the first draft refused (without draft: p
 * without d), or p of the last row when all are kept; also p where that
 * leaves nothing.  w_i counts in whole multiples of 2^-42 (rounded down,
 * values above 1 as 1, NaN as 0), so that its sums are exact in any order: the
 * token is the first whose inclusive sum exceeds floor(floor(pick 2^31) sum /
 * 2^31), or -1 where the row has no positive value.
 * Greedy: a draft is kept where it is the first largest value of its row (NaN
 * counts as the least; logits will do), and that of the next row follows.
 * A request without rows gets accepted 0.  A draft outside [0, V) is none: it is
 * refused, and the token after it is drawn from p, with nothing taken away.
 * Entries of emitted that belong to no request are not written.
 */
fk_status fk_verify(const fk_verify_args* a, void* ws, size_t ws_bytes, void* stream);

/* The pages of a pool as its rows hold them. */
typedef struct fk_kv_pool {
    int64_t R;             /* rows of the table, <= 2^20 */
    int64_t max_pages;
    int64_t pages;         /* of the pool */
    int32_t page_size;
    int32_t reserved;      /* 0 */
    int32_t* block_table;  /* [R][max_pages] */
    int32_t* lens;         /* [R] tokens of each row */
    int32_t* shares;       /* [pages] rows that hold a page, beyond the first;
                              0 for pages in the list */
    int32_t* free_pages;   /* [pages] the list of free pages */
    int32_t* free_count;   /* [1] */
} fk_kv_pool;

/* Bytes of workspace for n pairs on this pool (0 when invalid; only R,
 * max_pages, pages and page_size are looked at). */
size_t fk_kv_fork_workspace_bytes(int64_t n, const fk_kv_pool* p);

/*
 * fk_kv_fork -- row rows[i] becomes the first keep[i] tokens of row
 * sources[i], for all i at once: each sees the rows as they were before.
 * sources NULL: of itself, which returns its later tokens (keep 0: all).
 *   - Whole pages are shared and counted in shares.  The last, partly filled
 *     page is where the row goes on writing: it is kept by the one row that
 *     holds it when it was in no other row's reach, else it is copied to a
 *     page of the list.  copies[i] = (source page, destination page, tokens),
 *     or (-1, -1, 0); the caller has fk_kv4_copy move them, in every cache
 *     that the table serves, before the pages are written again.
 *   - Pages that no row holds any more go to the end of the list, in the
 *     order of the pairs and of their rows, before pages are taken: the last
 *     ones of the list, in its order, one for each copy in the order of the
 *     pairs.  If there are too few, the last copies are not made: those rows
 *     end with their last whole page, and lens says so.
 *   - A row named twice takes its first source and its least keep; rows
 *     outside [0, R) are none; a source outside is empty; lengths below 0
 *     are 0.  Entries of the table that the row loses become -1; rows that
 *     stay as they are are not touched.
 *   - seq [R] or NULL: of rows that change, their new length.
 * n <= 65536.  n * max_pages <= 2^31 - 1.
 */
fk_status fk_kv_fork(const fk_kv_pool* p, int64_t n, const int32_t* rows, const int32_t* sources,
                     const int32_t* keep, int32_t* copies, int32_t* seq, void* ws,
                     size_t ws_bytes, void* stream);

/* Bytes of workspace for fk_kv_compact of a pool of so many pages. */
size_t fk_kv_compact_workspace_bytes(int64_t pages);

/*
 * fk_kv_compact -- gives the U pages that are not in the list the numbers 0
 * .. U - 1: the k-th page in use from U on becomes the k-th free one below U.
 * Writes the table (entries below ceil(lens / page_size) are renamed, others
 * copied), shares, the list (its length in free_left, pages in descending
 * order so that the lowest are taken first; entries behind are not written)
 * and moves [n_moves] as fk_kv4_copy takes them, padded with (-1, -1, 0).
 * Each output may be its input.  n_moves >= pages / 2; pages <= 2^20.
 */
fk_status fk_kv_compact(const fk_kv_pool* p, int32_t* new_table, int32_t* new_shares,
                        int32_t* new_free, int32_t* free_left, int32_t* moves, int64_t n_moves,
                        void* ws, size_t ws_bytes, void* stream);

/*
 * fk_kv4_copy -- codes and scales of pages to other pages of the same cache:
 * of entry (source, destination, tokens) the blocks of 32 tokens that hold
 * the first `tokens`, of all heads.  Entries with a page outside the cache or
 * no tokens are skipped.  No page may be both source and destination of one
 * call, or destination twice.  n <= 2^20.
 */
fk_status fk_kv4_copy(const fk_kv4_cache* c, int64_t n, const int32_t* copies, void* stream);

/* Bytes of workspace for fk_kv4_attention_shared on any block table and window, of
 * up to B requests and so many groups; and of up to T tokens and max_q where
 * max_q q_heads / kv_heads is at most 48 (16 for 256 dimensions), else of T tokens
 * and this max_q.  0 when invalid. */
size_t fk_kv4_attn_shared_workspace_bytes(const fk_kv4_cache* c, int64_t B, int64_t T,
                                          int32_t q_heads, int32_t max_q, int64_t groups);

/*
 * fk_kv4_attention_shared -- fk_kv4_attention of requests that share their
 * first tokens.  Group g is the requests cu_groups[g] .. cu_groups[g+1] - 1
 * (ascending, else nothing is shared; requests of no group share nothing), of which the first
 * prefix_lens[g] tokens are the same: they are read through the row of the
 * table of the group's first request, once for the query rows of all of them.
 * Tokens behind the prefix's last whole block of 32 are read for each request.
 * out and lse are those of fk_kv4_attention up to the order of fp32 sums, and
 * its limits apply; groups <= B.  It pays for prefixes that are long beside the
 * requests' own tokens and the table's room: who shares is decided before
 * prefix_lens can be read, as if they filled max_pages, and short prefixes in a
 * wide table may take two to three times as long as fk_kv4_attention.
 */
fk_status fk_kv4_attention_shared(const fk_kv4_cache* c, const fk_kv4_attn* a, int64_t groups,
                                  const int32_t* cu_groups, const int32_t* prefix_lens, void* ws,
                                  size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FK_SERVE_H */
