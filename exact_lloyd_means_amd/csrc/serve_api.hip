// serve_api.hip -- host side of include/fk_serve.h: argument checks (before
// anything is enqueued) and workspace layouts.
#include <math.h>

#include "serve_internal.h"

namespace {

using namespace fk;

bool aligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

fk_status need(const void* p, const char* name, unsigned to) {
    if (!p) return fail(FK_EINVAL, "%s is NULL", name);
    if (!aligned(p, to)) return fail(FK_EINVAL, "%s is not %u-byte aligned", name, to);
    return FK_OK;
}

fk_status need_ws(const void* ws, size_t have, size_t want) {
    if (!ws) return fail(FK_EWORKSPACE, "workspace is NULL");
    if (!aligned(ws, 16)) return fail(FK_EINVAL, "workspace is not 16-byte aligned");
    if (have < want) return fail(FK_EWORKSPACE, "workspace has %zu bytes, needs %zu", have, want);
    return FK_OK;
}

#define FK_CHECK(expr)                    \
    do {                                  \
        fk_status fk_s_ = (expr);         \
        if (fk_s_ != FK_OK) return fk_s_; \
    } while (0)

constexpr int64_t kMaxRequests = 1 << 20, kMaxTokens = 1 << 24;

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

fk_status check_dtype(int32_t dtype) {
    if (dtype != FK_F32 && dtype != FK_F16 && dtype != FK_BF16)
        return fail(FK_EUNSUPPORTED, "dtype must be fp32, fp16 or bf16, got %d", (int)dtype);
    return FK_OK;
}

// ---- rotary positions --------------------------------------------------------------------

// Whether two of T x H rows of D elements share one: rows (dt, dh) apart start
// dt token - dh head elements apart.
bool rows_overlap(int64_t T, int64_t token, int64_t H, int64_t head, int64_t D) {
    if (H == 1) return T > 1 && token < D;
    if (T == 1) return head < D;
    if (token < D || head < D) return true;
    typedef __int128 wide;
    // rows of a token, or of a head, lie together: those of fused projections, of
    // either order of the dimensions
    if (token >= (wide)head * (H - 1) + D || head >= (wide)token * (T - 1) + D) return false;
    // else every distance of heads against the nearest two of tokens
    for (int64_t h = 1; h < H; ++h) {
        const wide at = (wide)head * h, t = at / token;
        if (t < T && at - t * token < D) return true;
        if (t + 1 < T && (t + 1) * token - at < D) return true;
    }
    return false;
}

// ---- verification -----------------------------------------------------------------------

fk_status check_verify_sizes(int64_t B, int64_t T, int64_t V) {
    if (B < 1 || T < 1 || V < 1)
        return fail(FK_EINVAL, "sizes must be >= 1 (B=%lld T=%lld V=%lld)", (long long)B,
                    (long long)T, (long long)V);
    if (B > kMaxRequests) return fail(FK_EUNSUPPORTED, "B must be <= 2^20");
    if (T > kMaxTokens) return fail(FK_EUNSUPPORTED, "T must be <= 2^24");
    if (V > 1 << 20) return fail(FK_EUNSUPPORTED, "V must be <= 2^20");
    return FK_OK;
}

// Elements of a piece of a row where `rows` of them are read: whole 16-byte
// accesses, and then the pieces that are left.
void cut_rows(int64_t rows, int64_t V, bool greedy, int32_t& pieces, int32_t& len) {
    const int64_t c = verify_pieces(rows, V, greedy);
    len = (int32_t)(((V + c - 1) / c + 7) / 8 * 8);
    pieces = (int32_t)((V + len - 1) / len);
}

// ---- pages --------------------------------------------------------------------------------

fk_status check_pool_sizes(const fk_kv_pool* p) {
    if (!p) return fail(FK_EINVAL, "pool is NULL");
    if (p->R < 1 || p->max_pages < 1 || p->pages < 1)
        return fail(FK_EINVAL, "sizes must be >= 1 (R=%lld max_pages=%lld pages=%lld)",
                    (long long)p->R, (long long)p->max_pages, (long long)p->pages);
    if (p->R > kMaxRequests) return fail(FK_EUNSUPPORTED, "R must be <= 2^20");
    if (p->page_size < 32 || p->page_size > 1024 || p->page_size % 32)
        return fail(FK_EUNSUPPORTED, "page_size must be a multiple of 32 up to 1024, got %d",
                    (int)p->page_size);
    if (p->max_pages > 2147483647 / p->page_size)
        return fail(FK_EUNSUPPORTED, "max_pages * page_size must be <= 2^31 - 1");
    if (p->pages > 2147483647 / p->page_size)
        return fail(FK_EUNSUPPORTED, "pages * page_size must be <= 2^31 - 1");
    if (p->reserved) return fail(FK_EINVAL, "reserved must be 0");
    return FK_OK;
}

fk_status check_pool(const fk_kv_pool* p) {
    FK_CHECK(check_pool_sizes(p));
    FK_CHECK(need(p->block_table, "block_table", 4));
    FK_CHECK(need(p->lens, "lens", 4));
    FK_CHECK(need(p->shares, "shares", 4));
    FK_CHECK(need(p->free_pages, "free_pages", 4));
    return need(p->free_count, "free_count", 4);
}

fk_status check_pairs(int64_t n, const fk_kv_pool* p) {
    if (n < 1) return fail(FK_EINVAL, "n must be >= 1");
    if (n > 65536) return fail(FK_EUNSUPPORTED, "n must be <= 65536");
    if (p->max_pages > 2147483647 / n)
        return fail(FK_EUNSUPPORTED, "n * max_pages must be <= 2^31 - 1");
    return FK_OK;
}

// Places in the workspace; base NULL: sizes only.
size_t fork_layout(int64_t n, const fk_kv_pool* p, char* base, ForkArgs& a) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* x = base ? base + at : nullptr;
        at = align256(at + bytes);
        return x;
    };
    a.info = reinterpret_cast<int32_t*>(take((size_t)n * 8 * sizeof(int32_t)));
    a.fresh = reinterpret_cast<int32_t*>(take((size_t)n * (size_t)p->max_pages * sizeof(int32_t)));
    a.have = reinterpret_cast<int32_t*>(take(2 * sizeof(int32_t)));
    a.count = reinterpret_cast<int32_t*>(take((size_t)p->pages * sizeof(int32_t)));
    a.tail = reinterpret_cast<int32_t*>(take((size_t)p->pages * sizeof(int32_t)));
    a.next = reinterpret_cast<int32_t*>(take((size_t)p->pages * sizeof(int32_t)));
    a.first = reinterpret_cast<uint64_t*>(take((size_t)p->pages * sizeof(uint64_t)));
    a.named = a.upto = nullptr;
    if (n >= kForkMany) {
        a.named = reinterpret_cast<int32_t*>(take((size_t)p->R * 2 * sizeof(int32_t)));
        a.upto = reinterpret_cast<int32_t*>(take((size_t)n * 2 * sizeof(int32_t)));
    }
    return at;
}

fk_status check_compact_pages(int64_t pages) {
    if (pages < 1) return fail(FK_EINVAL, "pages must be >= 1");
    if (pages > 1 << 20) return fail(FK_EUNSUPPORTED, "pages must be <= 2^20");
    return FK_OK;
}

size_t compact_layout(int64_t pages, char* base, CompactArgs& a) {
    const size_t words = (size_t)(pages + 31) / 32;
    a.bits = reinterpret_cast<uint32_t*>(base);
    const size_t at = align256(words * sizeof(uint32_t));
    a.before = base ? reinterpret_cast<int32_t*>(base + at) : nullptr;
    return at + (words + 1) * sizeof(int32_t);
}

// ---- attention of shared prefixes ------------------------------------------------------

// Workgroups of a head that run at once, two a CU.
int64_t shared_round(int Hkv) { return 512 / Hkv < 1 ? 1 : 512 / Hkv; }

// Places of a plan's sums in the workspace.
void shared_places(SharedPlan& p, int64_t B, int Hkv, int D) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t x = at;
        at = align256(at + bytes);
        return x;
    };
    const size_t units = (size_t)B * p.row_tiles, own = (size_t)Hkv * (units + 8 * (size_t)p.wgs) * p.rows;
    const size_t parts = (size_t)Hkv * (size_t)p.wgs * 16 * p.group_cols;
    p.head = take(16);
    p.unit = take(units * 48);
    p.part_o = take(parts * D * 4);
    p.part_ml = take(parts * 8);
    p.own_o = take(own * D * 4);
    p.own_ml = take(own * 8);
    p.total = at;
}

SharedPlan plan_shared(int64_t B, int64_t T, int Hq, int Hkv, int D, int max_q, int64_t groups,
                       int64_t room, int window) {
    SharedPlan p{};
    const int64_t G = Hq / Hkv, rows = G * max_q;
    const int most_cols = tile_cols(D), nb = rows <= 16 || most_cols == 1 ? 1 : 2;
    p.col_blocks = nb;
    const int64_t tiles = (rows + 16 * nb - 1) / (16 * nb);
    p.row_tiles = (int)tiles;
    // Tiles of a group of mean size: those that take the least time in all, which
    // for a block of 16 n rows goes as 3 + 5 n.
    const int64_t mean = (T * G + groups - 1) / groups;
    int64_t group_time = 0;
    for (int n = most_cols; n >= nb; --n) {
        if (nb == 2 && n < 3) break;
        const int64_t t = (mean + 16 * n - 1) / (16 * n) * (3 + 5 * n);
        if (!p.group_cols || t < group_time) {
            p.group_cols = n;
            group_time = t;
        }
    }
    const int na = p.group_cols;
    // Two workgroups a CU run at once; every tile of a group needs one, and one is
    // left.  A tile's segments are a workgroup's each, so tiles that leave much of
    // the card empty are better cut for two rounds, unless they are so short that
    // starting again (15 us) costs more.
    const int64_t most = T * G / (16 * na) + groups, round = shared_round(Hkv);
    int64_t seen = room;
    const int64_t behind = ((int64_t)window + max_q) / kKvBlock + 2;
    if (window > 0 && seen > behind) seen = behind;
    const double wide = D == 64 ? 0.6 : D == 128 ? 1.0 : 2.2;  // of a block's time
    int64_t rounds = most / round + 1;
    auto time = [&](int64_t r) {
        const int64_t segs = r * round / (most + 1);
        return (double)r * (150 + wide * (3 + 5 * na) * (double)((seen + 4 * segs - 1) / (4 * segs)));
    };
    if (rounds == 1 && most > round / 4 && time(2) < time(1)) rounds = 2;
    const int64_t wgs = rounds * round;
    p.use = groups <= kSharedGroups && B <= 8192 && room <= 1 << 22 && tiles * Hkv <= 65535 &&
            (room + kSharedUnit) * tiles <= (1 << 27) / B;
    // enough rows for the plain form's waves over rows, which beat both
    const int64_t row_wg = 64 * row_cols(D);
    p.use = p.use && (rows <= 16 * most_cols || (T * G + row_wg - 1) / row_wg * Hkv < 512);
    if (p.use) {
        // What sharing saves, in tenths of a microsecond of a wave, were all of the
        // table's room (or the window) the prefix, against the 8 us that finding
        // out who does what costs the walk, or 15 where the plain form is one launch.
        // That is right where prefixes fill much of the room: of 400 mixes of groups
        // of one to seven query tokens, in tables cut to the longest request, 59 are
        // shared, 47 of them gain (at most 82 us, 124 -> 41; 571 in all) and 11 lose
        // (at most 36, 111 -> 147; 71 in all).  With room for 131072 tokens 261 of the
        // same are shared, 81 gain (671 in all) and 165 lose (4 at the median, at most
        // 72, 94 -> 166; 1009 in all): how long prefixes are is not known here.
        const int64_t plain_cols = (rows + 15) / 16 < most_cols ? (rows + 15) / 16 : most_cols;
        const int64_t plain_time = (rows + 16 * plain_cols - 1) / (16 * plain_cols) * (3 + 5 * plain_cols);
        const double full = (double)wgs / (double)(wgs / (most + 1) * (most + 1));
        const double saved =
            wide * ((double)(B * plain_time) - (double)(groups * group_time) * full) * Hkv * (double)seen;
        // the requests' own keys as units of shares, where the plain form has no units
        const double units = wide * (double)(B * tiles * kSharedUnit * (nb == 1 ? 13 : 3 + 5 * nb)) * Hkv;
        p.use = room <= 64 ? saved - units >= 3e5 : saved >= 9e4;
    }
    if (!p.use) return p;
    p.rows = (int)(rows < 16 * nb ? rows : 16 * nb);
    // Least of a share: see the split form; and what a unit costs beside its blocks
    // (two blocks more: 64 groups of 4 96 -> 93 us, 16 of 16 54 -> 55, others alike).
    p.least = p.rows / 2 < kSharedUnit ? kSharedUnit : p.rows / 2;
    p.wgs = (int)wgs;
    const int64_t tiles_all = B * Hkv * tiles;
    int64_t z = 1024 / tiles_all;
    z = z < 1 ? 1 : z > p.rows ? p.rows : z;
    p.join_z = (int)z;
    const int each = (int)((p.rows + z - 1) / z), fit = 1024 / D;
    p.join_rows = 1;
    while (p.join_rows < each && p.join_rows < fit) p.join_rows *= 2;
    shared_places(p, B, Hkv, D);
    return p;
}

// Most bytes that plan_shared takes on any table and window for up to B requests
// and so many groups; and for up to T tokens and max_q where a request's rows fit
// a tile, else for those.
size_t shared_most(int64_t B, int64_t T, int Hq, int Hkv, int D, int max_q, int64_t groups) {
    const int64_t G = Hq / Hkv, rows = G * max_q;
    const int most_cols = tile_cols(D);
    groups = groups < kSharedGroups ? groups : kSharedGroups;
    B = B < 8192 ? B : 8192;
    size_t most = 0;
    auto form = [&](int64_t tokens, int64_t rows, int nb, int na) {
        const int64_t tiles = (rows + 16 * nb - 1) / (16 * nb), held = (1 << 27) / kSharedUnit / tiles;
        if (tiles * Hkv > 65535 || held < 1) return;
        SharedPlan p{};
        p.row_tiles = (int)tiles;
        p.rows = (int)(rows < 16 * nb ? rows : 16 * nb);
        p.group_cols = na;
        const int64_t n = tokens * G / (16 * na) + groups, round = shared_round(Hkv);
        // fewer tiles never take more rounds, but those above a quarter may take two
        const int64_t rounds = n < round && n > round / 4 ? 2 : n / round + 1;
        p.wgs = (int)(rounds * round);
        shared_places(p, B < held ? B : held, Hkv, D);
        most = most > p.total ? most : p.total;
    };
    // Rows of a tile of one block: groups of a mean of up to 16 rows have tiles of
    // one block (8 against 13 and 18 for two and three), and above 576 none has two
    // (13 ceil(m / 32) >= 18 ceil(m / 48)).
    auto blocks = [&](int64_t tokens, int64_t rows) {
        for (int na = 1; na <= most_cols; ++na) {
            const int64_t mean = na == most_cols ? T * G : na == 1 ? 16 : 576, fit = mean * groups / G;
            form(na < most_cols && fit < tokens ? fit : tokens, rows, 1, na);
        }
    };
    if (rows <= 16) {
        blocks(T, rows);
        return most;
    }
    const int64_t row_wg = 64 * row_cols(D);
    if (rows <= 16 * most_cols || (T * G + row_wg - 1) / row_wg * Hkv < 512)
        form(T, rows, most_cols == 1 ? 1 : 2, most_cols);
    if (rows <= 16 * most_cols && G <= 16) blocks(T, 16 / G * G);
    return most;
}

fk_status check_groups(int64_t groups, int64_t B) {
    if (groups < 1 || groups > B) return fail(FK_EINVAL, "groups must be 1 to B");
    return FK_OK;
}

}  // namespace

extern "C" {

fk_status fk_rope(const fk_rope_args* p, int32_t n, const fk_rope_rows* rows, void* stream) {
    if (!p || !rows) return fail(FK_EINVAL, "arguments are NULL");
    if (n != 1 && n != 2) return fail(FK_EINVAL, "n must be 1 or 2");
    if (p->T < 1) return fail(FK_EINVAL, "T must be >= 1");
    if (p->T > kMaxTokens) return fail(FK_EUNSUPPORTED, "T must be <= 2^24");
    FK_CHECK(check_dtype(p->dtype));
    if (p->head_dim < 2 || p->head_dim % 2 || p->head_dim > 1024)
        return fail(FK_EUNSUPPORTED, "head_dim must be even, 2 to 1024, got %d", (int)p->head_dim);
    if (p->rot_dim < 2 || p->rot_dim % 2 || p->rot_dim > p->head_dim)
        return fail(FK_EINVAL, "rot_dim must be even, 2 to head_dim, got %d", (int)p->rot_dim);
    if ((p->interleaved != 0 && p->interleaved != 1) || (p->inverse != 0 && p->inverse != 1))
        return fail(FK_EINVAL, "interleaved and inverse must be 0 or 1");
    if (!isfinite(p->factor)) return fail(FK_EINVAL, "factor must be finite");
    FK_CHECK(need(p->positions, "positions", 4));
    FK_CHECK(need(p->turns, "turns", 8));
    RopeArgs a{};
    const unsigned size = p->dtype == FK_F32 ? 4 : 2;
    for (int i = 0; i < n; ++i) {
        const fk_rope_rows& r = rows[i];
        if (r.heads < 1) return fail(FK_EINVAL, "heads must be >= 1");
        if (r.heads > 65536) return fail(FK_EUNSUPPORTED, "heads must be <= 2^16");
        FK_CHECK(need(r.x, "x", size));
        FK_CHECK(need(r.y, "y", size));
        if (r.x_token < 0 || r.x_head < 0 || r.y_token < 0 || r.y_head < 0)
            return fail(FK_EINVAL, "strides must be >= 0");
        if (r.x == r.y && (r.x_token != r.y_token || r.x_head != r.y_head))
            return fail(FK_EINVAL, "rows rotated in place must have the same strides");
        if (rows_overlap(p->T, r.y_token, r.heads, r.y_head, p->head_dim))
            return fail(FK_EINVAL, "rows of y overlap (strides %lld, %lld of %lld tokens, %d heads of %d)",
                        (long long)r.y_token, (long long)r.y_head, (long long)p->T, (int)r.heads,
                        (int)p->head_dim);
        if (i && r.y == rows[0].y) return fail(FK_EINVAL, "both sets have the same rows of y");
        if (r.reserved) return fail(FK_EINVAL, "reserved must be 0");
        a.set[i] = {r.x, r.y, r.x_token, r.x_head, r.y_token, r.y_head};
        a.heads[i] = r.heads;
    }
    if (n == 1) a.set[1] = a.set[0];  // without heads
    a.T = p->T;
    a.D = p->head_dim;
    a.R = p->rot_dim;
    a.pos = p->positions;
    a.turns = p->turns;
    a.factor = p->factor;
    a.sin_factor = p->inverse ? -p->factor : p->factor;
    const hipError_t e = launch_rope(a, p->dtype, p->interleaved, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? FK_OK : hip_fail(e, "fk_rope");
}

size_t fk_verify_workspace_bytes(int64_t B, int64_t T, int64_t V) {
    if (check_verify_sizes(B, T, V) != FK_OK) return 0;
    const size_t sampling = (size_t)verify_most_pieces(B, V, false) * 2;
    const size_t greedy = (size_t)verify_most_pieces(T, V, true);
    return (sampling > greedy ? sampling : greedy) * sizeof(uint64_t) + (size_t)B * sizeof(int32_t);
}

fk_status fk_verify(const fk_verify_args* p, void* ws, size_t ws_bytes, void* stream) {
    if (!p) return fail(FK_EINVAL, "arguments are NULL");
    FK_CHECK(check_verify_sizes(p->B, p->T, p->V));
    FK_CHECK(check_dtype(p->dtype));
    if (p->reserved) return fail(FK_EINVAL, "reserved must be 0");
    const unsigned size = p->dtype == FK_F32 ? 4 : 2;
    FK_CHECK(need(p->cu, "cu", 4));
    FK_CHECK(need(p->tokens, "tokens", 4));
    FK_CHECK(need(p->target, "target", size));
    if (p->draft) FK_CHECK(need(p->draft, "draft", size));
    if (p->target_row < 0 || p->draft_row < 0) return fail(FK_EINVAL, "strides must be >= 0");
    if (p->accept) {
        FK_CHECK(need(p->accept, "accept", 4));
        FK_CHECK(need(p->pick, "pick", 4));
    } else if (p->pick || p->draft) {
        return fail(FK_EINVAL, "pick and draft come with accept: greedy decoding draws nothing");
    }
    FK_CHECK(need(p->accepted, "accepted", 4));
    FK_CHECK(need(p->emitted, "emitted", 4));
    if (p->keep) {
        FK_CHECK(need(p->keep, "keep", 4));
        FK_CHECK(need(p->seq_lens, "seq_lens", 4));
    }
    FK_CHECK(need_ws(ws, ws_bytes, fk_verify_workspace_bytes(p->B, p->T, p->V)));
    // a request's drafts are read while tokens before them are written
    if (p->emitted == p->tokens) return fail(FK_EINVAL, "emitted must not be tokens");
    VerifyArgs a{};
    a.B = p->B;
    a.T = p->T;
    a.V = p->V;
    a.cu = p->cu;
    a.tokens = p->tokens;
    a.seq = p->seq_lens;
    a.p = p->target;
    a.q = p->draft;
    a.p_row = p->target_row;
    a.q_row = p->draft_row;
    a.u = p->accept;
    a.pick = p->pick;
    a.accepted = p->accepted;
    a.emitted = p->emitted;
    a.keep = p->keep;
    cut_rows(p->accept ? p->B : p->T, p->V, !p->accept, a.pieces, a.len);
    a.sums = static_cast<uint64_t*>(ws);
    a.kept = reinterpret_cast<int32_t*>(a.sums + p->B * a.pieces * 2);  // sampling only
    const hipError_t e = launch_verify(a, p->dtype, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? FK_OK : hip_fail(e, "fk_verify");
}

size_t fk_kv_fork_workspace_bytes(int64_t n, const fk_kv_pool* p) {
    if (check_pool_sizes(p) != FK_OK || check_pairs(n, p) != FK_OK) return 0;
    ForkArgs a{};
    return fork_layout(n, p, nullptr, a);
}

fk_status fk_kv_fork(const fk_kv_pool* p, int64_t n, const int32_t* rows, const int32_t* sources,
                     const int32_t* keep, int32_t* copies, int32_t* seq, void* ws,
                     size_t ws_bytes, void* stream) {
    FK_CHECK(check_pool(p));
    FK_CHECK(check_pairs(n, p));
    FK_CHECK(need(rows, "rows", 4));
    if (sources) FK_CHECK(need(sources, "sources", 4));
    FK_CHECK(need(keep, "keep", 4));
    FK_CHECK(need(copies, "copies", 4));
    if (seq) FK_CHECK(need(seq, "seq", 4));
    FK_CHECK(need_ws(ws, ws_bytes, fk_kv_fork_workspace_bytes(n, p)));
    ForkArgs a{};
    fork_layout(n, p, static_cast<char*>(ws), a);
    a.R = p->R;
    a.M = p->max_pages;
    a.N = p->pages;
    a.n = (int32_t)n;
    a.P = p->page_size;
    a.rows = rows;
    a.sources = sources;
    a.keep = keep;
    a.table = p->block_table;
    a.lens = p->lens;
    a.shares = p->shares;
    a.free_pages = p->free_pages;
    a.free_count = p->free_count;
    a.copies = copies;
    a.seq = seq;
    const hipError_t e = launch_kv_fork(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? FK_OK : hip_fail(e, "fk_kv_fork");
}

size_t fk_kv_compact_workspace_bytes(int64_t pages) {
    if (check_compact_pages(pages) != FK_OK) return 0;
    CompactArgs a{};
    return compact_layout(pages, nullptr, a);
}

fk_status fk_kv_compact(const fk_kv_pool* p, int32_t* new_table, int32_t* new_shares,
                        int32_t* new_free, int32_t* free_left, int32_t* moves, int64_t n_moves,
                        void* ws, size_t ws_bytes, void* stream) {
    FK_CHECK(check_pool(p));
    FK_CHECK(check_compact_pages(p->pages));
    FK_CHECK(need(new_table, "new_table", 4));
    FK_CHECK(need(new_shares, "new_shares", 4));
    FK_CHECK(need(new_free, "new_free", 4));
    FK_CHECK(need(free_left, "free_left", 4));
    if (n_moves < p->pages / 2) return fail(FK_EINVAL, "n_moves must be >= pages / 2");
    if (n_moves > 1 << 20) return fail(FK_EUNSUPPORTED, "n_moves must be <= 2^20");
    if (n_moves > 0) FK_CHECK(need(moves, "moves", 4));
    FK_CHECK(need_ws(ws, ws_bytes, fk_kv_compact_workspace_bytes(p->pages)));
    CompactArgs a{};
    compact_layout(p->pages, static_cast<char*>(ws), a);
    a.R = p->R;
    a.M = p->max_pages;
    a.N = p->pages;
    a.n_moves = n_moves;
    a.P = p->page_size;
    a.table = p->block_table;
    a.lens = p->lens;
    a.shares = p->shares;
    a.free_pages = p->free_pages;
    a.free_count = p->free_count;
    a.new_table = new_table;
    a.new_shares = new_shares;
    a.new_free = new_free;
    a.free_left = free_left;
    a.moves = moves;
    const hipError_t e = launch_kv_compact(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? FK_OK : hip_fail(e, "fk_kv_compact");
}

fk_status fk_kv4_copy(const fk_kv4_cache* c, int64_t n, const int32_t* copies, void* stream) {
    FK_CHECK(kv4_check_cache(c));
    if (n < 1) return fail(FK_EINVAL, "n must be >= 1");
    if (n > 1 << 20) return fail(FK_EUNSUPPORTED, "n must be <= 2^20");
    FK_CHECK(need(copies, "copies", 4));
    CopyArgs a{};
    a.codes = static_cast<uint8_t*>(c->codes);
    a.scales = static_cast<uint16_t*>(c->scales);
    a.copies = copies;
    a.pages = c->pages;
    a.n = (int32_t)n;
    a.P = c->page_size;
    a.H = c->kv_heads;
    a.D = c->head_dim;
    const hipError_t e = launch_kv4_copy(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? FK_OK : hip_fail(e, "fk_kv4_copy");
}

size_t fk_kv4_attn_shared_workspace_bytes(const fk_kv4_cache* c, int64_t B, int64_t T,
                                          int32_t q_heads, int32_t max_q, int64_t groups) {
    size_t plain = fk_kv4_attn_workspace_bytes(c, B, T, q_heads, max_q);
    if (!plain || check_groups(groups, B) != FK_OK) return 0;
    const int G = q_heads / c->kv_heads, q = (int)(T < max_q ? T : max_q);
    if (G <= 16 && G * q > 16 && G * q <= 16 * tile_cols(c->head_dim)) {
        // rows that fit a block: twice the waves
        const size_t few = fk_kv4_attn_workspace_bytes(c, B, T, q_heads, 16 / G);
        plain = plain > few ? plain : few;
    }
    const size_t most = shared_most(B, T, q_heads, c->kv_heads, c->head_dim, q, groups);
    return most > plain ? most : plain;
}

fk_status fk_kv4_attention_shared(const fk_kv4_cache* c, const fk_kv4_attn* p, int64_t groups,
                                  const int32_t* cu_groups, const int32_t* prefix_lens, void* ws,
                                  size_t ws_bytes, void* stream) {
    AttnArgs a;
    FK_CHECK(kv4_attn_args(c, p, a));
    FK_CHECK(check_groups(groups, p->B));
    FK_CHECK(need(cu_groups, "cu_groups", 4));
    FK_CHECK(need(prefix_lens, "prefix_lens", 4));
    const SharedPlan plan = plan_shared(p->B, p->T, p->q_heads, c->kv_heads, c->head_dim, a.max_q, groups,
                                        p->max_pages * (c->page_size / kKvBlock), p->window);
    if (!plan.use) return fk_kv4_attention(c, p, ws, ws_bytes, stream);
    FK_CHECK(need_ws(ws, ws_bytes, plan.total));
    char* w = static_cast<char*>(ws);
    a.least = plan.least;
    a.row_tiles = plan.row_tiles;
    a.part_rows = plan.rows;
    a.join_rows = plan.join_rows;
    a.part_o = reinterpret_cast<float*>(w + plan.part_o);
    a.part_ml = reinterpret_cast<float*>(w + plan.part_ml);
    SharedArgs s{};
    s.cu_groups = cu_groups;
    s.prefix = prefix_lens;
    s.groups = (int32_t)groups;
    s.wgs = plan.wgs;
    s.head = reinterpret_cast<int32_t*>(w + plan.head);
    s.unit = reinterpret_cast<int4*>(w + plan.unit);
    s.own_o = reinterpret_cast<float*>(w + plan.own_o);
    s.own_ml = reinterpret_cast<float*>(w + plan.own_ml);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const hipError_t e = c->head_dim == 64    ? launch_kv4_shared_d64(a, s, plan, c->dtype, st)
                         : c->head_dim == 128 ? launch_kv4_shared_d128(a, s, plan, c->dtype, st)
                                              : launch_kv4_shared_d256(a, s, plan, c->dtype, st);
    return e == hipSuccess ? FK_OK : hip_fail(e, "fk_kv4_attention_shared");
}

}  // extern "C"
