// kv4_api.hip -- host side of include/fk_kv4.h: argument checks (before
// anything is enqueued), workspace layout and the form a call runs.
#include <math.h>

#include "kv4_internal.h"

namespace fk {

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Workgroups that run at once: two of 80 KB of LDS on each of 256 CUs.
constexpr int kResident = 512;

AttnPlan plan_attention(int64_t B, int64_t T, int Hq, int Hkv, int D, int max_q,
                        int64_t max_blocks) {
    AttnPlan p{};
    const int64_t G = Hq / Hkv, rows = G * max_q;
    p.col_blocks = (int)((rows + 15) / 16 < tile_cols(D) ? (rows + 15) / 16 : tile_cols(D));
    const int64_t tile = 16 * p.col_blocks;
    const int64_t tiles = (rows + tile - 1) / tile;
    // Waves over rows need no join, but a card full of rows; below that the
    // keys are split.
    const int64_t wg = 64 * row_cols(D), row_wgs = (T * G + wg - 1) / wg * Hkv;
    p.split = (rows <= tile || row_wgs < kResident) && tiles * Hkv <= 65535;
    p.row_tiles = p.split ? (int)tiles : 1;
    p.rows = (int)(rows < tile ? rows : tile);
    // Where the table has room for few blocks a request, the longest decides,
    // and no launch that joins shares is worth its 8 us: one wave a request
    // where those alone nearly fill the card and are short (about 20 blocks is
    // where one and several meet), else as many as fit at once.  Measured with 8
    // kv heads of 128 alone, the longest request in blocks, us as one wave /
    // several / shares: 256 requests of 2: 10 / 13 / 24; 256 of 19: 27 / 27 /
    // 37; 128 of 32: 42 / 26 / 30; 128 of 63: 84 / 41 / 44; 16 of 32: - / 12 /
    // 20; 4 of 63: - / 16 / 19; 4 of 125: - / 26 / 21.
    if (p.split) {
        const int W = split_waves(D, p.col_blocks);
        const int64_t units = B * Hkv * tiles;
        int g = W;
        while (g > 1 && units * g > (int64_t)kResident * W) g /= 2;
        if (units >= 1024 && max_blocks <= 20) g = 1;
        const int64_t steps = (max_blocks + g - 1) / g;
        if (max_blocks <= 64 && steps * (D > 128 ? 2 : 1) <= 20) p.group = g;
    }
    if (p.split && !p.group) {
        // The join's workgroups, of 1024 / D rows at a time: about four a CU.
        const int64_t tiles_all = B * Hkv * tiles;
        int64_t z = 1024 / tiles_all;
        z = z < 1 ? 1 : z > p.rows ? p.rows : z;
        p.join_z = (int)z;
        const int each = (int)((p.rows + z - 1) / z), most = 1024 / D;
        p.join_rows = 1;
        while (p.join_rows < each && p.join_rows < most) p.join_rows *= 2;
        // Workgroups in whole rounds of the card: the fewest rounds of which
        // 88 % are full.
        const int64_t y = Hkv * tiles;
        double best = 0;
        for (int rounds = 1; rounds <= 8 && best < 0.88; ++rounds) {
            const int64_t s = rounds * kResident / y;
            const double full = (double)(s * y) / (rounds * kResident);
            if (full > best) {
                best = full;
                p.splits = (int)s;
            }
        }
        if (p.splits < 1) p.splits = 1;
        // A share's results are rows x D fp32, a block's codes and scales 32 D +
        // 128 bytes: at least a block for every two rows.
        p.least = p.rows / 2;
        const size_t waves = (size_t)p.splits * split_waves(D, p.col_blocks);
        const size_t parts = (size_t)Hkv * p.row_tiles * waves * 2 * (size_t)p.rows;
        size_t o = 0;
        p.part_o = o;
        o = align256(o + parts * D * sizeof(float));
        p.part_ml = o;
        o = align256(o + parts * 2 * sizeof(float));
        p.prefix = o;
        o = align256(o + (size_t)p.row_tiles * (size_t)(B + 1) * sizeof(int32_t));
        p.total = o;
    }
    if (p.total < 256) p.total = 256;
    return p;
}

}  // namespace fk

namespace {

using namespace fk;

bool aligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

fk_status need(const void* p, const char* name, unsigned to) {
    if (!p) return fail(FK_EINVAL, "%s is NULL", name);
    if (!aligned(p, to)) return fail(FK_EINVAL, "%s is not %u-byte aligned", name, to);
    return FK_OK;
}

#define FK_CHECK(expr)                    \
    do {                                  \
        fk_status fk_s_ = (expr);         \
        if (fk_s_ != FK_OK) return fk_s_; \
    } while (0)

constexpr int64_t kMaxRequests = 1 << 20;
constexpr int64_t kMaxTokens = 1 << 24;

fk_status check_page_size(int64_t P) {
    if (P < 32 || P > 1024 || P % 32)
        return fail(FK_EUNSUPPORTED, "page_size must be a multiple of 32 up to 1024, got %lld",
                    (long long)P);
    return FK_OK;
}

fk_status check_shape(const fk_kv4_cache* c) {
    if (!c) return fail(FK_EINVAL, "cache is NULL");
    if (c->pages < 1 || c->kv_heads < 1)
        return fail(FK_EINVAL, "sizes must be >= 1 (pages=%lld kv_heads=%d)", (long long)c->pages,
                    (int)c->kv_heads);
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return fail(FK_EUNSUPPORTED, "head_dim must be 64, 128 or 256, got %d", (int)c->head_dim);
    FK_CHECK(check_page_size(c->page_size));
    if (c->kv_heads > 1024) return fail(FK_EUNSUPPORTED, "kv_heads must be <= 1024");
    if (c->pages > 2147483647 / c->page_size)
        return fail(FK_EUNSUPPORTED, "pages * page_size must be <= 2^31 - 1");
    if (c->dtype != FK_F16 && c->dtype != FK_BF16)
        return fail(FK_EUNSUPPORTED, "cache dtype must be fp16 or bf16, got %d", (int)c->dtype);
    return FK_OK;
}

fk_status check_cache(const fk_kv4_cache* c) {
    FK_CHECK(check_shape(c));
    FK_CHECK(need(c->codes, "codes", 16));
    FK_CHECK(need(c->scales, "scales", 16));
    return need(c->codebook, "codebook", 16);
}

fk_status check_tokens(int64_t T) {
    if (T < 1) return fail(FK_EINVAL, "T must be >= 1");
    if (T > kMaxTokens) return fail(FK_EUNSUPPORTED, "T must be <= 2^24");
    return FK_OK;
}

fk_status check_rows(int64_t T, const fk_kv4_cache* c) {
    FK_CHECK(check_tokens(T));
    if (T * c->kv_heads > (int64_t)1 << 27)
        return fail(FK_EUNSUPPORTED, "T * kv_heads must be <= 2^27");
    return FK_OK;
}

fk_status check_requests(int64_t B) {
    if (B < 1) return fail(FK_EINVAL, "B must be >= 1");
    if (B > kMaxRequests) return fail(FK_EUNSUPPORTED, "B must be <= 2^20");
    return FK_OK;
}

fk_status check_strides(const char* name, int64_t token, int64_t head) {
    if (token < 0 || head < 0) return fail(FK_EINVAL, "strides of %s must be >= 0", name);
    return FK_OK;
}

// ceil(2^32 / d): the high half of x times it is x / d while x d < 2^32.  (d = 1
// does not fit; the kernels do not divide then.)
uint32_t division_magic(uint32_t d) { return (uint32_t)((((uint64_t)1 << 32) + d - 1) / d); }

// Rows that can be read in whole 16-byte pieces.
bool vec_rows(const void* p, int64_t token, int64_t head) {
    return aligned(p, 16) && token % 8 == 0 && head % 8 == 0;
}

RowArgs row_args(const fk_kv4_cache* c, int64_t T, const int32_t* slots) {
    RowArgs a{};
    a.codes = static_cast<uint8_t*>(c->codes);
    a.scales = static_cast<uint16_t*>(c->scales);
    a.codebook = static_cast<const uint16_t*>(c->codebook);
    a.slots = slots;
    a.T = T;
    a.slots_total = c->pages * c->page_size;
    a.page_size = c->page_size;
    a.H = c->kv_heads;
    a.bpp = (uint32_t)(c->page_size / kKvBlock);
    a.bpp_magic = division_magic(a.bpp);
    return a;
}

fk_status check_heads(const fk_kv4_cache* c, int64_t B, int64_t T, int32_t q_heads, int32_t max_q) {
    if (q_heads < 1 || q_heads % c->kv_heads)
        return fail(FK_EINVAL, "q_heads (%d) must be a multiple of kv_heads (%d)", (int)q_heads,
                    (int)c->kv_heads);
    if (q_heads / c->kv_heads > 256) return fail(FK_EUNSUPPORTED, "q_heads / kv_heads must be <= 256");
    if (T * (q_heads / c->kv_heads) > kMaxTokens)
        return fail(FK_EUNSUPPORTED, "T * q_heads / kv_heads must be <= 2^24");
    if (((T * (q_heads / c->kv_heads) + 63) / 64 + B) * c->kv_heads >= (int64_t)1 << 24)
        return fail(FK_EUNSUPPORTED, "T * q_heads / 64 + B * kv_heads must be < 2^24");
    if (max_q < 1) return fail(FK_EINVAL, "max_q must be >= 1");
    return FK_OK;
}

// No request has more query tokens than there are.
int clamp_max_q(int64_t T, int32_t max_q) { return T < max_q ? (int)T : max_q; }

}  // namespace

namespace fk {
fk_status kv4_check_cache(const fk_kv4_cache* c) { return check_cache(c); }

fk_status kv4_attn_args(const fk_kv4_cache* c, const fk_kv4_attn* p, AttnArgs& a) {
    FK_CHECK(check_cache(c));
    if (!p) return fail(FK_EINVAL, "arguments are NULL");
    FK_CHECK(check_requests(p->B));
    FK_CHECK(check_tokens(p->T));
    FK_CHECK(check_heads(c, p->B, p->T, p->q_heads, p->max_q));
    if (p->max_pages < 1) return fail(FK_EINVAL, "max_pages must be >= 1");
    if (p->max_pages > 2147483647 / c->page_size)
        return fail(FK_EUNSUPPORTED, "max_pages * page_size must be <= 2^31 - 1");
    if (p->max_pages * (c->page_size / kKvBlock) > 2147483647 / p->B)
        return fail(FK_EUNSUPPORTED, "B * max_pages * page_size must be < 2^36");
    if (!(p->scale > 0.f) || !isfinite(p->scale))
        return fail(FK_EINVAL, "scale must be positive and finite");
    if (p->causal != 0 && p->causal != 1) return fail(FK_EINVAL, "causal must be 0 or 1");
    if (p->window < 0) return fail(FK_EINVAL, "window must be >= 0");
    FK_CHECK(need(p->q, "q", 2));
    FK_CHECK(check_strides("q", p->q_token, p->q_head));
    FK_CHECK(need(p->cu_q, "cu_q", 4));
    FK_CHECK(need(p->seq_lens, "seq_lens", 4));
    FK_CHECK(need(p->block_table, "block_table", 4));
    FK_CHECK(need(p->out, "out", 16));
    if (p->lse) FK_CHECK(need(p->lse, "lse", 4));
    a = AttnArgs{};
    a.codes = static_cast<const uint8_t*>(c->codes);
    a.scales = static_cast<const uint16_t*>(c->scales);
    a.codebook = static_cast<const uint16_t*>(c->codebook);
    a.q = static_cast<const uint16_t*>(p->q);
    a.out = static_cast<uint16_t*>(p->out);
    a.lse = p->lse;
    a.cu = p->cu_q;
    a.seq = p->seq_lens;
    a.table = p->block_table;
    a.q_token = p->q_token;
    a.q_head = p->q_head;
    a.T = p->T;
    a.max_pages = p->max_pages;
    a.pages = c->pages;
    a.B = (int32_t)p->B;
    a.Hq = p->q_heads;
    a.Hkv = c->kv_heads;
    a.G = p->q_heads / c->kv_heads;
    a.page_size = c->page_size;
    a.causal = p->causal;
    a.window = p->window;
    a.max_q = clamp_max_q(p->T, p->max_q);
    a.q_vec = vec_rows(p->q, p->q_token, p->q_head);
    a.bpp = (uint32_t)(c->page_size / kKvBlock);
    a.bpp_magic = division_magic(a.bpp);
    a.G_magic = division_magic((uint32_t)a.G);
    a.cap = (int32_t)(p->max_pages * c->page_size);
    a.qk = p->scale * 1.4426950408889634f;
    return FK_OK;
}
}  // namespace fk

extern "C" {

size_t fk_kv_plan_workspace_bytes(int64_t B) {
    if (check_requests(B) != FK_OK) return 0;
    return (size_t)(B + 1) * sizeof(int32_t);
}

fk_status fk_kv_plan(int64_t B, int64_t max_pages, int32_t page_size, const int32_t* ctx_lens,
                     const int32_t* new_lens, const int32_t* free_pages, int64_t free_cap,
                     const int32_t* free_count, int32_t* block_table, int32_t* seq_lens,
                     int32_t* cu_new, int32_t* slots, int32_t* positions, int64_t slot_cap,
                     int32_t* free_left, int32_t* status, void* ws, size_t ws_bytes,
                     void* stream) {
    return fk_kv_plan_kept(B, max_pages, page_size, ctx_lens, new_lens, free_pages, free_cap,
                           free_count, block_table, seq_lens, cu_new, slots, positions, slot_cap,
                           free_left, status, nullptr, ws, ws_bytes, stream);
}

fk_status fk_kv_plan_kept(int64_t B, int64_t max_pages, int32_t page_size, const int32_t* ctx_lens,
                          const int32_t* new_lens, const int32_t* free_pages, int64_t free_cap,
                          const int32_t* free_count, int32_t* block_table, int32_t* seq_lens,
                          int32_t* cu_new, int32_t* slots, int32_t* positions, int64_t slot_cap,
                          int32_t* free_left, int32_t* status, int32_t* kept_lens, void* ws,
                          size_t ws_bytes, void* stream) {
    FK_CHECK(check_requests(B));
    FK_CHECK(check_page_size(page_size));
    if (max_pages < 1 || free_cap < 0 || slot_cap < 0)
        return fail(FK_EINVAL, "max_pages must be >= 1, free_cap and slot_cap >= 0");
    if (max_pages > 2147483647 || free_cap > 2147483647 || slot_cap > 2147483647)
        return fail(FK_EUNSUPPORTED, "max_pages, free_cap and slot_cap must be <= 2^31 - 1");
    FK_CHECK(need(ctx_lens, "ctx_lens", 4));
    FK_CHECK(need(new_lens, "new_lens", 4));
    if (free_cap > 0) FK_CHECK(need(free_pages, "free_pages", 4));
    FK_CHECK(need(free_count, "free_count", 4));
    FK_CHECK(need(block_table, "block_table", 4));
    FK_CHECK(need(seq_lens, "seq_lens", 4));
    FK_CHECK(need(cu_new, "cu_new", 4));
    if (slot_cap > 0) FK_CHECK(need(slots, "slots", 4));
    if (positions) FK_CHECK(need(positions, "positions", 4));
    FK_CHECK(need(free_left, "free_left", 4));
    FK_CHECK(need(status, "status", 4));
    if (kept_lens) FK_CHECK(need(kept_lens, "kept_lens", 4));
    if (!ws) return fail(FK_EWORKSPACE, "workspace is NULL");
    if (!aligned(ws, 16)) return fail(FK_EINVAL, "workspace is not 16-byte aligned");
    const size_t bytes = fk_kv_plan_workspace_bytes(B);
    if (ws_bytes < bytes)
        return fail(FK_EWORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, bytes);
    PlanArgs a{};
    a.B = B;
    a.max_pages = max_pages;
    a.free_cap = free_cap;
    a.slot_cap = slot_cap;
    a.page_size = page_size;
    a.ctx = ctx_lens;
    a.fresh = new_lens;
    a.free_pages = free_pages;
    a.free_count = free_count;
    a.table = block_table;
    a.seq = seq_lens;
    a.cu = cu_new;
    a.slots = slots;
    a.pos = positions;
    a.free_left = free_left;
    a.status = status;
    a.kept = kept_lens;
    a.ws = static_cast<int32_t*>(ws);
    const hipError_t e = launch_kv_plan(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? FK_OK : hip_fail(e, "fk_kv_plan");
}

fk_status fk_kv4_write(const fk_kv4_cache* c, int64_t T, const void* k, int64_t k_token,
                       int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                       const int32_t* slots, void* stream) {
    FK_CHECK(check_cache(c));
    FK_CHECK(check_rows(T, c));
    FK_CHECK(need(k, "k", 2));
    FK_CHECK(need(v, "v", 2));
    FK_CHECK(check_strides("k", k_token, k_head));
    FK_CHECK(check_strides("v", v_token, v_head));
    FK_CHECK(need(slots, "slots", 4));
    RowArgs a = row_args(c, T, slots);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.k_token = k_token;
    a.k_head = k_head;
    a.v_token = v_token;
    a.v_head = v_head;
    const bool vec = vec_rows(k, k_token, k_head) && vec_rows(v, v_token, v_head);
    const hipError_t e =
        launch_kv4_write(a, c->head_dim, c->dtype, vec, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? FK_OK : hip_fail(e, "fk_kv4_write");
}

fk_status fk_kv4_read(const fk_kv4_cache* c, int64_t T, const int32_t* slots, void* k, void* v,
                      void* stream) {
    FK_CHECK(check_cache(c));
    FK_CHECK(check_rows(T, c));
    FK_CHECK(need(slots, "slots", 4));
    FK_CHECK(need(k, "k", 16));
    FK_CHECK(need(v, "v", 16));
    RowArgs a = row_args(c, T, slots);
    a.ko = static_cast<uint16_t*>(k);
    a.vo = static_cast<uint16_t*>(v);
    const hipError_t e = launch_kv4_read(a, c->head_dim, c->dtype, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? FK_OK : hip_fail(e, "fk_kv4_read");
}

size_t fk_kv4_attn_workspace_bytes(const fk_kv4_cache* c, int64_t B, int64_t T, int32_t q_heads,
                                   int32_t max_q) {
    if (check_shape(c) != FK_OK || check_requests(B) != FK_OK || check_tokens(T) != FK_OK ||
        check_heads(c, B, T, q_heads, max_q) != FK_OK)
        return 0;
    // as much as a call with any block table needs
    return plan_attention(B, T, q_heads, c->kv_heads, c->head_dim, clamp_max_q(T, max_q),
                          (int64_t)1 << 40).total;
}

fk_status fk_kv4_attention(const fk_kv4_cache* c, const fk_kv4_attn* p, void* ws, size_t ws_bytes,
                           void* stream) {
    AttnArgs a;
    FK_CHECK(kv4_attn_args(c, p, a));
    const AttnPlan plan = plan_attention(p->B, p->T, p->q_heads, c->kv_heads, c->head_dim, a.max_q,
                                         p->max_pages * (c->page_size / kKvBlock));
    if (!ws) return fail(FK_EWORKSPACE, "workspace is NULL");
    if (!aligned(ws, 16)) return fail(FK_EINVAL, "workspace is not 16-byte aligned");
    if (ws_bytes < plan.total)
        return fail(FK_EWORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, plan.total);
    a.least = plan.least;
    a.group = plan.group;
    a.row_tiles = plan.row_tiles;
    a.splits = plan.splits;
    a.part_rows = plan.rows;
    a.join_rows = plan.join_rows;
    char* w = static_cast<char*>(ws);
    a.part_o = reinterpret_cast<float*>(w + plan.part_o);
    a.part_ml = reinterpret_cast<float*>(w + plan.part_ml);
    a.prefix = reinterpret_cast<int32_t*>(w + plan.prefix);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = c->head_dim == 64    ? launch_kv4_attn_d64(a, plan, c->dtype, s)
                         : c->head_dim == 128 ? launch_kv4_attn_d128(a, plan, c->dtype, s)
                                              : launch_kv4_attn_d256(a, plan, c->dtype, s);
    return e == hipSuccess ? FK_OK : hip_fail(e, "fk_kv4_attention");
}

}  // extern "C"
