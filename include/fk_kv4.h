/*
 * fk_kv4.h -- a paged key/value cache held as 4-bit codebook indices, for
 * AMD Instinct MI355X (gfx950): the plan of a serving step, rows written to
 * the cache and read back, and attention over it.
 *
 * Low-bit KV quantisation is one of the uses the pages name for exact
 * batched k-means (papernotes.org notes, 研究背景与动机; 7minutos.es article,
 * "Casos de uso"); a codebook here is the 16 centroids that fk_lloyd gives
 * for the normalised values of one head (K = 16, d = 1, B = heads).
 *
 * The cache
 * ---------
 *  Row      one token's k or v of one kv head, D = head_dim values x_i of
 *           the cache dtype (fp16 or bf16).  It is kept as its scale
 *             s = max_i |x_i|          (exact; NaN when a value is not finite)
 *           and D codes of 4 bits.  With c_0 <= ... <= c_15 the head's
 *           codebook and t_j = (c_j + c_{j+1}) / 2 rounded to fp16,
 *             code_i = number of j with t_j s < x_i,
 *           so a value on a threshold takes the lower code.  It stands for
 *             c_code s.
 *           t_j s has at most 22 bits and is exact in fp32 from s = 2^-118
 *           up (smaller bf16 scales may round): codes do not depend on
 *           rounding or order.
 *  codebook [2][kv_heads][16] fp16, k then v, each ascending and finite.
 *  scales   [pages][kv_heads][2][page_size] cache dtype.
 *  codes    [pages][kv_heads][2][page_size / 32][16 D] bytes: blocks of 32
 *           tokens in the operand order of the matrix instructions, so that
 *           a wave reads a block with whole 1 KB loads and no transposition
 *           through LDS.  A block is D/64 pieces of 64 lanes x 16 bytes
 *           (piece p, lane l, byte y at 1024 p + 16 l + y); lane l = 16 g + i
 *           owns D/4 bytes, byte a of them in piece a / 16:
 *             k  tokens t = 8 (i/4) + 4 tile + i%4 (tile 0, 1), dimensions
 *                g D/4 + w (w < D/4): byte tile D/8 + w/2;
 *             v  tokens t = 8 g + j (j < 8), dimensions i D/16 + w (w <
 *                D/16): byte 32 (w/8) + j min(4, D/32) + (w%8)/2.
 *           An even dimension is the low half of its byte.
 *  Slot     page * page_size + place in the page, as int32; negative: none.
 *
 * Conventions are those of fk.h (streams, workspaces, errors, nothing
 * allocated or kept), except where stated: int32 arrays need 4-byte
 * alignment, q, k and v 2-byte alignment; codes, scales, codebook, out and
 * workspaces 16-byte alignment.
 *  Limits   head_dim 64, 128 or 256; page_size a multiple of 32, at most
 *           1024; pages * page_size <= 2^31 - 1; kv_heads <= 1024; dtype
 *           FK_F16 or FK_BF16.
 */
#ifndef FK_KV4_H
#define FK_KV4_H

#include "fk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A cache: its storage (device pointers) and shape. */
typedef struct fk_kv4_cache {
    void* codes;
    void* scales;
    const void* codebook;
    int64_t pages;
    int32_t page_size, kv_heads, head_dim;
    int32_t dtype;
} fk_kv4_cache;

/* Bytes of workspace for fk_kv_plan of B requests (0 if B is invalid). */
size_t fk_kv_plan_workspace_bytes(int64_t B);

/*
 * fk_kv_plan -- block tables and slot maps of one step, from the lengths on
 * the GPU.  Request b holds ctx_lens[b] tokens and gets new_lens[b] more
 * (negative lengths count as 0).  With seq = ctx + new and held = ceil(ctx /
 * page_size) it needs the pages held .. min(ceil(seq / page_size),
 * max_pages) - 1 of its table.  Needed pages are numbered in request order;
 * number i takes free_pages[n - 1 - i], n = *free_count clamped to [0,
 * free_cap], or -1 when the list is spent.
 *   block_table [B][max_pages]  needed entries are written, others are not
 *                     touched; entries below held must be there;
 *   seq_lens [B]      seq;
 *   cu_new [B+1]      exclusive prefix sums of new;
 *   slots [slot_cap]  of new token i (requests in order): its slot, or -1
 *                     where it has no page, and for i >= cu_new[B];
 *   positions [slot_cap] its position in its request, -1 for i >= cu_new[B]
 *                     (may be NULL);
 *   free_left [1]     n minus the pages taken (may be free_count itself);
 *   status [4]        new tokens, pages taken, pages wanted but not there,
 *                     new tokens left without a page by the end of the list
 *                     or of the table.
 * Sums saturate at 2^31 - 1.  Tokens from slot_cap on get no slot; their
 * pages are taken all the same.  B <= 2^20, max_pages >= 1.
 */
fk_status fk_kv_plan(int64_t B, int64_t max_pages, int32_t page_size, const int32_t* ctx_lens,
                     const int32_t* new_lens, const int32_t* free_pages, int64_t free_cap,
                     const int32_t* free_count, int32_t* block_table, int32_t* seq_lens,
                     int32_t* cu_new, int32_t* slots, int32_t* positions, int64_t slot_cap,
                     int32_t* free_left, int32_t* status, void* ws, size_t ws_bytes, void* stream);

/*
 * fk_kv_plan_kept -- fk_kv_plan that also says what the next step's ctx_lens
 * are: kept_lens [B] (or NULL) is ctx plus the new tokens that have a page.
 * That is seq unless the list or the table ended.  The tokens after them have
 * no rows in the cache: entries below ceil(seq / page_size) are then missing
 * from the table, and a plan that took seq for ctx would never ask for them.
 */
fk_status fk_kv_plan_kept(int64_t B, int64_t max_pages, int32_t page_size, const int32_t* ctx_lens,
                          const int32_t* new_lens, const int32_t* free_pages, int64_t free_cap,
                          const int32_t* free_count, int32_t* block_table, int32_t* seq_lens,
                          int32_t* cu_new, int32_t* slots, int32_t* positions, int64_t slot_cap,
                          int32_t* free_left, int32_t* status, int32_t* kept_lens, void* ws,
                          size_t ws_bytes, void* stream);

/*
 * fk_kv4_write -- rows k, v of T tokens into the cache.  Element (t, h, i)
 * of k is at k[t * k_token + h * k_head + i] (strides in elements, >= 0),
 * of v likewise.  Tokens whose slot is negative or beyond the cache are
 * skipped; two tokens of one call must not share a slot.
 */
fk_status fk_kv4_write(const fk_kv4_cache* c, int64_t T, const void* k, int64_t k_token,
                       int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                       const int32_t* slots, void* stream);

/*
 * fk_kv4_read -- the rows of T slots as the values they stand for, rounded
 * to the cache dtype: k, v [T][kv_heads][head_dim].  Rows of slots that are
 * negative or beyond the cache are zeros.
 */
fk_status fk_kv4_read(const fk_kv4_cache* c, int64_t T, const int32_t* slots, void* k, void* v,
                      void* stream);

/* Attention over the cache: sizes, inputs and options. */
typedef struct fk_kv4_attn {
    int64_t B;             /* requests */
    int64_t T;             /* query tokens of all requests */
    int32_t q_heads;       /* a multiple of kv_heads */
    int32_t max_q;         /* most query tokens of one request, or more;
                              those of a request from max_q on are left out */
    int64_t max_pages;     /* row length of block_table */
    int64_t q_token, q_head; /* strides of q in elements */
    const void* q;         /* (T, q_heads, head_dim) in the cache dtype */
    const int32_t* cu_q;   /* [B+1] first query token of each request */
    const int32_t* seq_lens; /* [B] tokens of each request in the cache */
    const int32_t* block_table; /* [B][max_pages] */
    float scale;           /* factor of q.k, > 0 and finite */
    int32_t causal;        /* 1: query i of n sees positions <= seq - n + i */
    int32_t window;        /* > 0: and only positions > seq - n + i - window */
    void* out;             /* [T][q_heads][head_dim] cache dtype */
    float* lse;            /* [T][q_heads] or NULL */
} fk_kv4_attn;

/* Bytes of workspace for fk_kv4_attention; 0 when the arguments are invalid. */
size_t fk_kv4_attn_workspace_bytes(const fk_kv4_cache* c, int64_t B, int64_t T, int32_t q_heads,
                                   int32_t max_q);

/*
 * fk_kv4_attention -- softmax attention of the queries over the cached rows
 * of their requests.  Query token i of the n = cu_q[b+1] - cu_q[b] of
 * request b stands at position seq_lens[b] - n + i; head h reads kv head
 * h / (q_heads / kv_heads).  out = sum_j softmax_j(scale q.k_j) v_j over the
 * positions j it sees, lse = ln sum_j exp(scale q.k_j); a query that sees
 * nothing gives zeros and -inf.  Positions in pages that the table does not
 * name (entry outside [0, pages)) or beyond max_pages are not seen.  Rows of
 * out and lse that belong to no request, or to query tokens i >= max_q, are
 * not written.  Scores,
 * sums and the running maximum are fp32; the products run on fp16 matrix
 * instructions: q scaled by a power of two per row (exact for values down to
 * 2^-14 of the row's largest, in bf16 to 2^-17; below that to 2^-25 of the
 * largest), codebook values as they are, softmax weights times v's scale
 * rounded to fp16 once: to 2^-11 of the weight, or 2^-28 of the largest of
 * its row where that is more.  v scales below 2^-96 or above 2^40, which only
 * bf16 holds, may cost more, as may those above 2^15 beside scores beyond 2^24.
 * Results do not depend on timing.  B <= 2^20, q_heads / kv_heads <= 256, T *
 * q_heads / kv_heads <= 2^24, B * max_pages * page_size < 2^36, (ceil(T *
 * q_heads / kv_heads / 64) + B) * kv_heads < 2^24.
 */
fk_status fk_kv4_attention(const fk_kv4_cache* c, const fk_kv4_attn* a, void* ws, size_t ws_bytes,
                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FK_KV4_H */
