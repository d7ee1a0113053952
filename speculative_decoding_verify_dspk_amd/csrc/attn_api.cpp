// C ABI of the attention side of the pass: argument checks, launch plans and
// launches.  As in the rest of the ABI, everything the host can see is checked
// before anything is enqueued; nothing here allocates, frees or synchronises.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "../../include/dspk.h"
#include "attn_internal.h"
#include "dspk_internal.h"

namespace dspk {

AttnPlan attn_plan(int32_t q_heads, int32_t kv_heads, int32_t d, int32_t b, int32_t max_rows, int64_t capacity,
                   int cus) {
    AttnPlan p;
    const int64_t rows = (int64_t)max_rows * (q_heads / kv_heads);    // rows over one k/v head
    const int64_t tiles = (rows + 15) / 16;
    const int64_t unit = kAttnStep * kAttnWaves, per_seg = capacity < 1 ? 1 : (capacity + unit - 1) / unit;
    const int64_t segs = (int64_t)b * kv_heads;
    p.fits = segs <= INT32_MAX / per_seg;                             // segs * per_seg, without overflowing
    const int64_t units = p.fits ? segs * per_seg : INT32_MAX;
    // One row tile per wave where a CU gets few units: a launch of two is some 2
    // us slower before its first unit (twice the registers and LDS), but takes k
    // and v half as often.  One tile against two, by units x tiles per CU, caches
    // in memory, 8 k/v heads: 2 (16 rows of 32 heads, one request of 4000
    // positions, bf16) 13.3 against 14.9 us; 4 (6 rows, four of 4000) 21.6 against
    // 24.2; 8 (6 rows, four of 8000) 30.2 / 30.6, (16 rows, one of 16000) 30.5 /
    // 27.8; 12 (17 rows of 40 heads, one of 16000) 36.8 / 31.5; 16 (16 rows, one of
    // 32000) 47.0 / 38.4.  8 bits alike: 19.5 / 22.7 at 4, 42.9 / 34.0 at 16.
    const int most_tiles = attn_tiles(d);
    p.tiles = units <= 8 * (int64_t)cus / tiles ? 1 : most_tiles < tiles ? most_tiles : (int32_t)tiles;
    p.blocks = (int32_t)((tiles + p.tiles - 1) / p.tiles);
    const int32_t most = cus > p.blocks ? cus / p.blocks : 1;         // one workgroup per CU
    p.groups = (int32_t)(units < most ? units : most);
    p.pairs = per_seg == 2;                                           // tables of 257 .. 512 positions
    // The last group of a segment adds the pieces of all by itself, at the rate
    // of one CU; where they are many, a launch of its own is faster (one request
    // of 8 rows, two tiles, 4 / 8 / 32 pieces: 11.5 / 15 / 26 us in one launch, 12.7
    // / 12.7 / 13.5 us in two; one tile was not measured).  `pieces` is what lengths
    // that fill the page table would leave, or one more where ranges do not start with
    // a segment: shorter contexts pay for the launch without needing it (a tree of 16
    // over 1000 positions of a bf16 cache 9.0 us under a table of that size, 11.4
    // under 8 times it, 14.0 under 128 times it, with two tiles then).
    const int64_t pieces = segs >= p.groups ? 2 : per_seg < p.groups / segs ? per_seg : p.groups / segs + 1;
    p.join = pieces * p.tiles * 16 * d * (int64_t)sizeof(float) > kAttnJoinBytes;
    // The workspace is that of the most tiles, which no other choice exceeds: two
    // pieces per workgroup, of the segment it did not start and of the one it does
    // not end.
    const int64_t row_blocks = (tiles + most_tiles - 1) / most_tiles;
    const size_t wgs = cus > row_blocks ? cus : row_blocks;
    p.off_part = (2 * wgs * kAttnWaves * kAttnCounter * sizeof(uint32_t) + 255) / 256 * 256;
    p.ws_bytes = p.off_part + wgs * 2 * attn_piece(d, tiles < most_tiles ? 1 : most_tiles) * sizeof(float);
    p.ws_bytes = (p.ws_bytes + 255) / 256 * 256;
    return p;
}

RowsPlan rows_plan(const AttnBatch &B, int32_t heads, int32_t d, int32_t q_heads, bool read) {
    RowsPlan g{};
    // no request has more rows than the arrays hold; counted in 64 bits, for
    // max_rows and total_rows go up to 2^31 - 1
    int64_t rows = B.max_rows < B.total_rows ? B.max_rows : B.total_rows;
    rows = rows < 1 ? 1 : rows;
    // 2^bs positions that `rows` rows can touch, wherever they start
    const auto touched = [&](int bs) { return ((rows + (1 << bs) - 2) >> bs) + 1; };
    g.bs = kBlockShift;
    int64_t nb = touched(g.bs), kv = nb * B.b * heads;
    // Few blocks are halved, to double the workgroups at work: norm, rotation and
    // store of one request of 128 / 512 rows of 32 + 8 + 8 heads 9.9 / 10.7 -> 6.6 /
    // 7.2 us; more (960 of 64 positions, three prompts of 2500 rows) take 41.5 us
    // whole and 44.6 halved.
    if (!read && kv <= 512) {
        nb = touched(--g.bs);
        kv = nb * B.b * heads;
    }
    // q: few rows go one to a workgroup, sliced further into passes, for latency;
    // many in chunks (40 heads: 32 requests of 8 rows 7.2 us singly and 8.9 in
    // chunks, 512 rows 11.1 and 10.8, 2048 rows 17.7 and 14.4)
    const bool many = B.total_rows >= 1024;
    g.q_rows = many ? kManyQRows : 1;
    const int64_t q_blocks = (rows + g.q_rows - 1) / g.q_rows;
    g.slices = many ? 1 : ((int64_t)q_heads * d + kRowThreads * 8 - 1) / (kRowThreads * 8);
    const int64_t q = q_heads == 0 ? 0 : B.b * q_blocks * g.slices;
    g.fits = kv <= kLaunchThreads / kRowThreads && q <= kLaunchThreads / kRowThreads - kv;
    if (!g.fits) return g;
    g.nb = (int32_t)nb;
    g.kv_blocks = (int32_t)kv;
    g.q_blocks = (int32_t)q_blocks;
    g.grid = (int32_t)(kv + q);
    return g;
}

}  // namespace dspk

namespace {

int fail(int code, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return dspk::set_error(code, buf);
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

int launch_result(hipError_t e, const char *who) {
    if (e != hipSuccess) return fail(DSPK_EDEVICE, "%s: launch failed: %s", who, hipGetErrorString(e));
    return dspk::set_error(DSPK_OK, "");
}

bool pointer(const void *p, size_t a) { return p != nullptr && aligned(p, a); }

int check_dim(int32_t d, const char *who) {
    if (d != 64 && d != 128 && d != 256)
        return fail(DSPK_EUNSUPPORTED, "%s: head_dim=%d (supported: 64, 128, 256)", who, d);
    return DSPK_OK;
}

// The format of a cache; its pointers are checked where they are used.
int check_format(const dspk_kv_cache *c, dspk::KvCache &out, const char *who) {
    if (c == nullptr) return fail(DSPK_EINVAL, "%s: cache descriptor is NULL", who);
    if (c->bits != 8 && c->bits != 16) return fail(DSPK_EUNSUPPORTED, "%s: cache bits=%d (supported: 8, 16)", who, c->bits);
    int rc = check_dim(c->head_dim, who);
    if (rc) return rc;
    if (c->kv_heads < 1 || c->kv_heads > 65535) return fail(DSPK_EINVAL, "%s: kv_heads=%d out of 1..65535", who, c->kv_heads);
    const int32_t pt = c->page_tokens;
    if (pt < dspk::kBlockTokens || pt > 65536 || (pt & (pt - 1)))
        return fail(DSPK_EUNSUPPORTED, "%s: page_tokens=%d (supported: powers of two, 64..65536)", who, pt);
    if (c->pages < 1 || c->pages > INT32_MAX) return fail(DSPK_EINVAL, "%s: pages=%lld out of 1..2^31-1", who, (long long)c->pages);
    out.heads = c->kv_heads;
    out.d = c->head_dim;
    out.bits = c->bits;
    out.page_shift = 0;
    while ((1 << out.page_shift) < pt) ++out.page_shift;
    out.pages = c->pages;
    return DSPK_OK;
}

int check_pools(const dspk_kv_cache *c, const char *who) {
    if (!pointer(c->k, 256) || !pointer(c->v, 256))
        return fail(DSPK_EINVAL, "%s: cache k and v must be non-NULL 256-byte aligned device pointers", who);
    if (c->bits == 8 && (!pointer(c->k_scales, 16) || !pointer(c->v_scales, 16)))
        return fail(DSPK_EINVAL, "%s: an 8-bit cache needs 16-byte aligned k_scales and v_scales", who);
    if (c->bits == 16 && (c->k_scales != nullptr || c->v_scales != nullptr))
        return fail(DSPK_EINVAL, "%s: a bf16 cache takes no scales", who);
    return DSPK_OK;
}

int check_cache(const dspk_kv_cache *c, dspk::KvCache &out, const char *who) {
    int rc = check_format(c, out, who);
    if (rc) return rc;
    rc = check_pools(c, who);
    if (rc) return rc;
    out.k = c->k;
    out.v = c->v;
    out.ks = c->k_scales;
    out.vs = c->v_scales;
    return DSPK_OK;
}

int check_batch(const dspk_attn_batch *B, const dspk::KvCache &c, dspk::AttnBatch &out, const char *who) {
    if (B == nullptr) return fail(DSPK_EINVAL, "%s: batch descriptor is NULL", who);
    if (B->b < 1 || B->b > 65535) return fail(DSPK_EINVAL, "%s: b=%d out of 1..65535", who, B->b);
    if (B->max_rows < 1) return fail(DSPK_EINVAL, "%s: max_rows=%d must be >= 1", who, B->max_rows);
    if (B->max_pages < 1) return fail(DSPK_EINVAL, "%s: max_pages=%d must be >= 1", who, B->max_pages);
    if (B->total_rows < 0 || (B->row_start == nullptr && (int64_t)B->b * B->max_rows > B->total_rows))
        return fail(DSPK_EINVAL, "%s: total_rows=%d holds fewer than b x max_rows rows", who, B->total_rows);
    if (!pointer(B->cache_len, 4) || !pointer(B->page_table, 4) || !aligned(B->row_start, 4))
        return fail(DSPK_EINVAL, "%s: cache_len or page_table NULL, or an array misaligned", who);
    // positions, and what the kernels add to them, stay within 31 bits
    if ((int64_t)B->max_pages << c.page_shift > 1 << 30)
        return fail(DSPK_EUNSUPPORTED, "%s: max_pages=%d of %d positions (at most 2^30 positions per request)", who,
                    B->max_pages, 1 << c.page_shift);
    out.b = B->b;
    out.max_rows = B->max_rows;
    out.total_rows = B->total_rows;
    out.max_pages = B->max_pages;
    out.row_start = B->row_start;
    out.cache_len = B->cache_len;
    out.page_table = B->page_table;
    return DSPK_OK;
}

// Row arrays [rows][ld]: 16-byte aligned rows of at least heads * d elements.
int check_rows(const void *p, int64_t ld, int32_t heads, int32_t d, int32_t dtype, const char *name, const char *who) {
    if (dtype != DSPK_F32 && dtype != DSPK_BF16) return fail(DSPK_EINVAL, "%s: bad element type %d", who, dtype);
    const int64_t per = dtype == DSPK_F32 ? 4 : 8;
    if (!pointer(p, 16)) return fail(DSPK_EINVAL, "%s: %s must be a non-NULL 16-byte aligned device pointer", who, name);
    if (ld < (int64_t)heads * d || ld % per)
        return fail(DSPK_EINVAL, "%s: leading dimension %lld of %s must be >= %lld and a multiple of %lld", who,
                    (long long)ld, name, (long long)heads * d, (long long)per);
    return DSPK_OK;
}

int check_rows_plan(const dspk::RowsPlan &g, const char *who) {
    if (!g.fits) return fail(DSPK_EUNSUPPORTED, "%s: too many rows for one launch", who);
    return DSPK_OK;
}

int append_common(const char *who, const dspk_kv_cache *cache, const dspk_attn_batch *batch, dspk::AppendArgs &A,
                  const void *k, int64_t ldk, const void *v, int64_t ldv, int32_t dtype, void *stream) {
    int rc = check_cache(cache, A.c, who);
    if (rc) return rc;
    rc = check_batch(batch, A.c, A.B, who);
    if (rc) return rc;
    rc = check_rows(k, ldk, A.c.heads, A.c.d, dtype, "k", who);
    if (rc) return rc;
    rc = check_rows(v, ldv, A.c.heads, A.c.d, dtype, "v", who);
    if (rc) return rc;
    A.g = dspk::rows_plan(A.B, A.c.heads, A.c.d, A.q == nullptr ? 0 : A.q_heads, false);
    rc = check_rows_plan(A.g, who);
    if (rc) return rc;
    A.k = k;
    A.v = v;
    A.ldk = ldk;
    A.ldv = ldv;
    A.f32 = dtype == DSPK_F32;
    return launch_result(dspk::launch_append(A, (hipStream_t)stream), who);
}

int check_tree(int32_t b, int32_t m_rows, const int32_t *parents, const char *who) {
    if (b < 1) return fail(DSPK_EINVAL, "%s: b=%d must be >= 1", who, b);
    if (m_rows < 1 || m_rows > DSPK_MAX_TREE)
        return fail(DSPK_EINVAL, "%s: m_rows=%d out of 1..%d", who, m_rows, DSPK_MAX_TREE);
    if (b > dspk::kLaunchThreads / 64) return fail(DSPK_EUNSUPPORTED, "%s: b=%d requests for one launch", who, b);
    if (m_rows > 1 && !pointer(parents, 4)) return fail(DSPK_EINVAL, "%s: parents NULL or misaligned", who);
    return DSPK_OK;
}

}  // namespace

extern "C" {

size_t dspk_kv_cache_bytes(int64_t pages, int32_t kv_heads, int32_t head_dim, int32_t page_tokens, int32_t bits) {
    dspk_kv_cache c = {kv_heads, head_dim, page_tokens, bits, pages, nullptr, nullptr, nullptr, nullptr};
    dspk::KvCache out;
    if (check_format(&c, out, "dspk_kv_cache_bytes")) return 0;
    const size_t positions = (size_t)pages * kv_heads, row = (size_t)page_tokens * head_dim * (bits / 8);
    return positions > SIZE_MAX / row ? 0 : positions * row;
}

int dspk_qkv_norm_rope_append(const dspk_kv_cache *cache, const dspk_attn_batch *batch, const dspk_qk_prep *prep,
                              const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                              int32_t dtype, int32_t q_heads, uint16_t *q_out, int64_t ldqo, void *stream) {
    const char *who = "dspk_qkv_norm_rope_append";
    if (prep == nullptr) return fail(DSPK_EINVAL, "%s: prep is NULL", who);
    if (cache == nullptr) return fail(DSPK_EINVAL, "%s: cache descriptor is NULL", who);
    int rc = check_dim(cache->head_dim, who);
    if (rc) return rc;
    const int32_t d = cache->head_dim;
    if (q_heads < 1 || q_heads > 65535) return fail(DSPK_EINVAL, "%s: q_heads=%d out of 1..65535", who, q_heads);
    rc = check_rows(q, ldq, q_heads, d, dtype, "q", who);
    if (rc) return rc;
    rc = check_rows(q_out, ldqo, q_heads, d, DSPK_BF16, "q_out", who);
    if (rc) return rc;
    if (!aligned(prep->q_weight, 16) || !aligned(prep->k_weight, 16))
        return fail(DSPK_EINVAL, "%s: norm weights must be 16-byte aligned", who);
    if ((prep->q_weight != nullptr || prep->k_weight != nullptr) && !(prep->eps >= 0.f && isfinite(prep->eps)))
        return fail(DSPK_EINVAL, "%s: eps must be finite and >= 0", who);
    if (prep->inv_freq != nullptr) {
        if (!aligned(prep->inv_freq, 4)) return fail(DSPK_EINVAL, "%s: inv_freq misaligned", who);
        if (prep->rotary_dim < 2 || prep->rotary_dim > d || prep->rotary_dim % 2)
            return fail(DSPK_EINVAL, "%s: rotary_dim=%d out of 2..%d, or odd", who, prep->rotary_dim, d);
        if (prep->rotary_dim % 16)
            return fail(DSPK_EUNSUPPORTED, "%s: rotary_dim=%d (supported: multiples of 16)", who, prep->rotary_dim);
        if (prep->interleaved != 0 && prep->interleaved != 1)
            return fail(DSPK_EINVAL, "%s: interleaved=%d (0 or 1)", who, prep->interleaved);
        if (!aligned(prep->positions, 4)) return fail(DSPK_EINVAL, "%s: positions misaligned", who);
    }
    if ((const void *)q_out == q && (dtype != DSPK_BF16 || ldqo != ldq))
        return fail(DSPK_EINVAL, "%s: q_out may be q only if q is bf16 with the same leading dimension", who);
    dspk::AppendArgs A{};
    A.q = q;
    A.ldq = ldq;
    A.q_heads = q_heads;
    A.q_out = q_out;
    A.ldqo = ldqo;
    A.eps = prep->eps;
    A.qw = prep->q_weight;
    A.kw = prep->k_weight;
    A.inv_freq = prep->inv_freq;
    A.rot = prep->rotary_dim;
    A.interleaved = prep->interleaved;
    A.positions = prep->positions;
    return append_common(who, cache, batch, A, k, ldk, v, ldv, dtype, stream);
}

int dspk_kv_append(const dspk_kv_cache *cache, const dspk_attn_batch *batch, const void *k, int64_t ldk, const void *v,
                   int64_t ldv, int32_t dtype, void *stream) {
    dspk::AppendArgs A{};
    return append_common("dspk_kv_append", cache, batch, A, k, ldk, v, ldv, dtype, stream);
}

int dspk_kv_read(const dspk_kv_cache *cache, const dspk_attn_batch *batch, void *k, int64_t ldk, void *v, int64_t ldv,
                 int32_t dtype, void *stream) {
    const char *who = "dspk_kv_read";
    dspk::ReadArgs A{};
    int rc = check_cache(cache, A.c, who);
    if (rc) return rc;
    rc = check_batch(batch, A.c, A.B, who);
    if (rc) return rc;
    rc = check_rows(k, ldk, A.c.heads, A.c.d, dtype, "k", who);
    if (rc) return rc;
    rc = check_rows(v, ldv, A.c.heads, A.c.d, dtype, "v", who);
    if (rc) return rc;
    A.g = dspk::rows_plan(A.B, A.c.heads, A.c.d, 0, true);
    rc = check_rows_plan(A.g, who);
    if (rc) return rc;
    A.k = k;
    A.v = v;
    A.ldk = ldk;
    A.ldv = ldv;
    A.f32 = dtype == DSPK_F32;
    return launch_result(dspk::launch_kv_read(A, (hipStream_t)stream), who);
}

size_t dspk_attn_workspace_bytes(int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t b, int32_t max_rows) {
    if (kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads || q_heads / kv_heads > 256 || b < 1 || max_rows < 1 ||
        max_rows > DSPK_MAX_TREE || (head_dim != 64 && head_dim != 128 && head_dim != 256))
        return 0;
    return dspk::attn_plan(q_heads, kv_heads, head_dim, b, max_rows, 1, dspk::device_cus()).ws_bytes;
}

int dspk_tree_attention(const dspk_kv_cache *cache, const dspk_attn_batch *batch, const uint16_t *q, int64_t ldq,
                        int32_t q_heads, float scale, const uint64_t *tree_mask, uint16_t *out, int64_t ldo,
                        void *workspace, size_t ws_bytes, void *stream) {
    const char *who = "dspk_tree_attention";
    dspk::AttnArgs A{};
    int rc = check_cache(cache, A.c, who);
    if (rc) return rc;
    rc = check_batch(batch, A.c, A.B, who);
    if (rc) return rc;
    if (A.B.max_rows > DSPK_MAX_TREE)
        return fail(DSPK_EUNSUPPORTED, "%s: max_rows=%d (at most %d rows of one request)", who, A.B.max_rows,
                    DSPK_MAX_TREE);
    if (q_heads < A.c.heads || q_heads % A.c.heads)
        return fail(DSPK_EINVAL, "%s: q_heads=%d must be a multiple of kv_heads=%d", who, q_heads, A.c.heads);
    if (q_heads / A.c.heads > 256)
        return fail(DSPK_EUNSUPPORTED, "%s: q_heads=%d (at most 256 per k/v head)", who, q_heads);
    rc = check_rows(q, ldq, q_heads, A.c.d, DSPK_BF16, "q", who);
    if (rc) return rc;
    rc = check_rows(out, ldo, q_heads, A.c.d, DSPK_BF16, "out", who);
    if (rc) return rc;
    if (!(scale > 0.f) || !isfinite(scale)) return fail(DSPK_EINVAL, "%s: scale must be finite and > 0", who);
    if (!aligned(tree_mask, 8)) return fail(DSPK_EINVAL, "%s: tree_mask misaligned", who);
    const dspk::AttnPlan p = dspk::attn_plan(q_heads, A.c.heads, A.c.d, A.B.b, A.B.max_rows,
                                             (int64_t)A.B.max_pages << A.c.page_shift, dspk::device_cus());
    if (!p.fits || (int64_t)A.c.heads * p.blocks > 65535) return fail(DSPK_EUNSUPPORTED, "%s: page table, or heads times rows, too large for one launch", who);
    if (!pointer(workspace, 256) || ws_bytes < p.ws_bytes)
        return fail(DSPK_EINVAL, "%s: workspace of %zu bytes required (256-byte aligned)", who, p.ws_bytes);
    if (q == out) return fail(DSPK_EINVAL, "%s: out must not be q", who);
    A.q = q;
    A.ldq = ldq;
    A.out = out;
    A.ldo = ldo;
    A.rep = q_heads / A.c.heads;
    A.scale = scale * 1.44269504088896340736f;
    A.mask = tree_mask;
    A.tiles = p.tiles;
    A.blocks = p.blocks;
    A.groups = p.groups;
    A.join = p.join;
    A.pairs = p.pairs;
    A.counters = (uint32_t *)workspace;
    A.part = (float *)((char *)workspace + p.off_part);
    return launch_result(dspk::launch_tree_attention(A, (hipStream_t)stream), who);
}

int dspk_tree_layout(const int32_t *parents, int32_t b, int32_t m_rows, const int32_t *cache_len, uint64_t *tree_mask,
                     int32_t *positions, void *stream) {
    const char *who = "dspk_tree_layout";
    int rc = check_tree(b, m_rows, parents, who);
    if (rc) return rc;
    if (!pointer(cache_len, 4) || !pointer(tree_mask, 8) || !pointer(positions, 4))
        return fail(DSPK_EINVAL, "%s: cache_len, tree_mask or positions NULL or misaligned", who);
    return launch_result(
        dspk::launch_tree_layout(parents, b, m_rows, cache_len, tree_mask, positions, (hipStream_t)stream), who);
}

int dspk_accept_tree_greedy(const int32_t *target_ids, const int32_t *draft_ids, const int32_t *parents, int32_t b,
                            int32_t m_rows, int32_t *accept_len, int32_t *committed, int32_t *path, void *stream) {
    const char *who = "dspk_accept_tree_greedy";
    int rc = check_tree(b, m_rows, parents, who);
    if (rc) return rc;
    if (!pointer(target_ids, 4) || !pointer(accept_len, 4) || !pointer(committed, 4) || !pointer(path, 4))
        return fail(DSPK_EINVAL, "%s: target_ids, accept_len, committed or path NULL or misaligned", who);
    if (m_rows > 1 && !pointer(draft_ids, 4)) return fail(DSPK_EINVAL, "%s: draft_ids NULL or misaligned", who);
    return launch_result(dspk::launch_accept_tree(target_ids, draft_ids, parents, b, m_rows, accept_len, committed, path,
                                                  (hipStream_t)stream),
                         who);
}

int dspk_kv_commit(int32_t count, const dspk_kv_cache *caches, const dspk_attn_batch *batch, const int32_t *path,
                   const int32_t *accept_len, int32_t *new_len, void *stream) {
    const char *who = "dspk_kv_commit";
    if (count < 1 || caches == nullptr) return fail(DSPK_EINVAL, "%s: count=%d caches, or NULL", who, count);
    dspk::CommitArgs A{};
    for (int32_t i = 0; i < count; ++i) {
        dspk::KvCache c;
        int rc = check_cache(&caches[i], c, who);
        if (rc) return rc;
        if (i == 0) A.c = c;
        if (c.heads != A.c.heads || c.d != A.c.d || c.bits != A.c.bits || c.page_shift != A.c.page_shift ||
            c.pages != A.c.pages)
            return fail(DSPK_EINVAL, "%s: caches of one call must have the same shape", who);
    }
    int rc = check_batch(batch, A.c, A.B, who);
    if (rc) return rc;
    if (A.B.row_start != nullptr || A.B.max_rows > DSPK_MAX_TREE)
        return fail(DSPK_EUNSUPPORTED, "%s: every request has max_rows nodes, at most %d (row_start must be NULL)", who,
                    DSPK_MAX_TREE);
    if (!pointer(path, 4) || !pointer(accept_len, 4) || !aligned(new_len, 4))
        return fail(DSPK_EINVAL, "%s: path or accept_len NULL, or an array misaligned", who);
    // workgroups read these after others have written new_len
    const auto over = [&](const int32_t *p, int64_t n) {
        const uintptr_t a = (uintptr_t)new_len, e = (uintptr_t)p;
        return new_len != nullptr && a < e + n * sizeof(int32_t) && e < a + A.B.b * sizeof(int32_t);
    };
    const bool in_place = new_len == A.B.cache_len;
    if (!in_place && over(A.B.cache_len, A.B.b))
        return fail(DSPK_EINVAL, "%s: new_len overlaps cache_len without being it", who);
    if (over(accept_len, A.B.b) || over(path, (int64_t)A.B.b * A.B.max_rows) ||
        (!in_place && over(A.B.page_table, (int64_t)A.B.b * A.B.max_pages)))
        return fail(DSPK_EINVAL, "%s: new_len overlaps accept_len, path or the page table", who);
    A.path = path;
    A.accept_len = accept_len;
    // a new_len that is cache_len is written by a launch of its own, after
    // every workgroup has read the old lengths
    for (int32_t i = 0; i < count; i += dspk::kMaxCaches) {
        A.count = count - i < dspk::kMaxCaches ? count - i : dspk::kMaxCaches;
        for (int32_t j = 0; j < A.count; ++j)
            A.caches[j] = {caches[i + j].k, caches[i + j].v, caches[i + j].k_scales, caches[i + j].v_scales};
        A.new_len = i == 0 && !in_place ? new_len : nullptr;
        const hipError_t e = dspk::launch_kv_commit(A, (hipStream_t)stream);
        if (e != hipSuccess) return launch_result(e, who);
    }
    if (in_place) {
        A.new_len = new_len;
        return launch_result(dspk::launch_new_len(A, (hipStream_t)stream), who);
    }
    return launch_result(hipSuccess, who);
}

}  // extern "C"
