// C ABI of the 8-bit integer side: argument checks, launch plans and launches.  As
// in the rest of the ABI, everything the host can see is checked before anything
// is enqueued; nothing here allocates, frees or synchronises.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "../../include/dspk.h"
#include "i8_internal.h"

namespace dspk {

// Which kernel a product takes.
//
// Streams read each weight fragment once into registers and all of x for every 16 or
// 32 columns: best while x is small beside the weight.  Tiles stage both through
// LDS, so x is read once per 64 to 256 columns.  Measured (us, weights in memory,
// tiles with their best splits of K), n x k:
//            4096x4096       2560x9728       19456x2560      5120x17408
//   rows   stream  tile    stream  tile    stream  tile    stream  tile
//      1     4.7    9.9      6.7   10.0      9.8   12.4     15.9   20.8
//     16     5.7   10.0      9.9   10.2     11.8   13.2     20.9   21.2
//     18     5.8   10.2     10.3   10.4     12.6   13.7     23.2   21.4
//     32     7.1   10.2     13.9   10.5     15.7   14.4     30.2   21.6
//     36     8.1    9.0     15.8   10.9     17.8   15.1     33.0   23.1
//     64    11.0    9.1     22.6   11.3     23.7   16.2     45.5   24.2
// Two column tiles per stream workgroup where there are more tiles than CUs (16
// rows, 384 tiles: 6.4 -> 5.8 us), one where there are not (160 tiles: 6.2 / 5.3).
//
// The choice is by estimates fitted to some 2000 measured launches of 170 products, 20
// to 3000 rows: it is .9% behind the best of them on average, 14% at worst.  A
// round of tiles takes 3.4 us and a time per stage of 128 K (1.55 times that for two
// workgroups on a CU), but no less than the weight's way from memory; a split 1.75 us and
// .35 us per MB of sums that change hands; a stream moves its columns and all rows of x
// past a CU at some 32 GB/s.
I8Plan i8_plan(int32_t n, int32_t k, int32_t m, bool split, int cus) {
    I8Plan p{};
    const int64_t steps = i8_steps(k), stages = steps / 2, tiles = i8_tiles(n);
    const auto over = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    p.splits = 1;
    struct Shape {
        I8Kind kind;
        int rows, cols;
        double own;                 // us of a stage alone on a CU; two share it in 1.55 times that
    };
    static const Shape shapes[] = {{kI8Tile32x64, 32, 64, .19}, {kI8Tile64x64, 64, 64, .225},
                                   {kI8Tile64x128, 64, 128, .345}, {kI8Tile128x128, 128, 128, .66}};
    double best = 1e300;
    for (const Shape &c : shapes) {
        if (m <= 16) break;
        if (m <= 32 ? c.rows != 32 : c.rows == 32) continue;
        const int64_t of = over(m, c.rows) * over(n, c.cols);
        for (int s = 1; s <= 8; ++s) {
            if (s > 1 && (!split || stages < 4 * s || of * s > 4 * cus || of > kI8MaxSplitTiles)) break;
            const int64_t all = of * s;
            const double stage = all > cus ? 1.55 * c.own : c.own;
            const double tiled = (double)over(all, 2 * cus) * (3.4 + (double)stages / s * stage);
            const double read = 3.4 + 1e-6 / 7.3 * n * k;
            const double us = (tiled > read ? tiled : read) + (s > 1 ? 1.75 + .35e-6 * 4 * all * c.rows * c.cols : 0);
            if (us >= best) continue;
            best = us;
            p.kind = c.kind;
            p.splits = s;
            p.groups = of;
            p.off_part = p.ws_bytes = 0;
            if (s > 1) {
                p.off_part = kMoeHead;
                p.ws_bytes = p.off_part + (size_t)all * c.rows * c.cols * sizeof(int32_t);
            }
        }
    }
    const bool wide = tiles > cus;
    const int64_t groups = over(tiles, wide ? 2 : 1);
    if (m <= 16 || (m <= 64 && 1.4 + 31e-6 * (m + (wide ? 32 : 16)) * k * over(groups, cus) <= best)) {
        p = I8Plan{};
        p.splits = 1;
        p.kind = m <= 16 ? (wide ? kI8Stream16x2 : kI8Stream16x1)
                 : m <= 32 ? (wide ? kI8Stream32x2 : kI8Stream32x1) : (wide ? kI8Stream64x2 : kI8Stream64x1);
        // 4 to 7 waves (8 never have fewer turns than 4 have), so that their rings' last
        // turns are full (40 fragments, rings of 4: 5 waves 11.9 us, 4 12.7)
        const int ring = p.kind == kI8Stream16x1 ? 8 : p.kind == kI8Stream64x2 ? 2 : 4;
        int64_t least = INT64_MAX;
        for (int w = 4; w <= 7; ++w) {
            const int64_t turns = over(steps, (int64_t)w * ring) * w * ring;
            if (turns < least) least = turns, p.waves = w;
        }
        p.groups = groups;
        p.fits = p.groups * 64 * p.waves <= UINT32_MAX;
        return p;
    }
    // 256 x 256: whole rounds of one workgroup per CU, then the rest in quarters, if that
    // is the shorter
    const int64_t big = over(m, 256) * over(n, 256), rest = big % cus;
    const double whole = 8 + 1.5 * stages, quarters = (double)over(4 * rest, cus) * (4 + .5 * stages);
    const bool cut = rest != 0 && quarters < whole;
    const double us = (double)(cut ? big / cus : over(big, cus)) * whole + (cut ? quarters : 0);
    if (m > 64 && us < best) {
        p = I8Plan{};
        p.kind = kI8Tile256x256;
        p.splits = 1;
        p.whole = cut ? big - rest : big;
        p.groups = p.whole + 4 * (big - p.whole);
    }
    p.fits = p.groups * 512 <= UINT32_MAX;
    return p;
}

MoePlan moe_plan(int32_t hidden, int32_t inter, int32_t experts, int32_t m, int32_t top_k, int cus) {
    MoePlan p{};
    const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    const size_t slots = (size_t)m * top_k;
    p.ldh = ((int64_t)inter + kI8Cols - 1) / kI8Cols * kI8Cols;
    p.off_scores = up(kMoeHead);
    p.off_h = up(p.off_scores + (size_t)m * experts * sizeof(float));
    p.off_h8 = up(p.off_h + slots * p.ldh * sizeof(float));
    p.off_h_scales = up(p.off_h8 + slots * p.ldh);
    p.off_top = up(p.off_h_scales + slots * sizeof(float));
    p.off_part = up(p.off_top + slots * (p.ldh / kI8Cols) * sizeof(uint32_t));
    // h's codes made by each down workgroup, a row per wave: the layer's two launches (2048
    // columns) for 8 slots of 768 values 17.6 -> 14.6 us, of 1536 23.4 -> 20.7, of 2048 27.1 -> 24.8, of
    // 4096 42.5 -> 42.1; for 2 slots of 2048 15.6 -> 13.7, of 4096 21.1 -> 20.1 (4096 columns 27.4 ->
    // 28.3), but of 14336 46.6 -> 56.4, which a wave alone turns into codes.
    p.inside = slots <= kDownWaves && p.ldh <= kMoeInside;
    // Enough workgroups for the CUs, where one group of slots is all and each wave keeps
    // two pieces of work or more (2048 columns, 8 / 16 / 48 slots of 768, both launches: one
    // part 14.6 / 21.8 / 48.6 us, two 15.8 / 22.0 / 42.9, four 19.7 / 25.7 / 46.3).
    const int64_t tiles = i8_tiles(hidden), work = ((int64_t)slots < experts ? (int64_t)slots : experts) * ((i8_steps(inter) + 7) / 8);
    p.parts = 1;
    if (slots <= kMoeGroup && tiles <= kMoeSplitTiles)
        while (p.parts < kMoeMaxParts && tiles * p.parts * 2 <= cus && work >= 32 * p.parts) p.parts *= 2;
    p.ws_bytes = up(p.off_part + (p.parts > 1 ? tiles * p.parts * slots * 16 * sizeof(int32_t) : 0));
    return p;
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

int ok() { return dspk::set_error(DSPK_OK, ""); }

int launch_result(hipError_t e, const char *who) {
    if (e != hipSuccess) return fail(DSPK_EDEVICE, "%s: launch failed: %s", who, hipGetErrorString(e));
    return ok();
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool pointer(const void *p, size_t a) { return p != nullptr && aligned(p, a); }

int check_dtype(int32_t dtype, const char *name, const char *who) {
    if (dtype != DSPK_F32 && dtype != DSPK_BF16)
        return fail(DSPK_EINVAL, "%s: element type %d of %s (DSPK_F32 or DSPK_BF16)", who, dtype, name);
    return DSPK_OK;
}

// Rows [m][ld] of n elements, in whole 16-byte pieces.
int check_rows(const void *p, int64_t ld, int32_t n, int32_t dtype, const char *name, const char *who) {
    const int64_t per = dtype == DSPK_F32 ? 4 : 8;
    if (!pointer(p, 16)) return fail(DSPK_EINVAL, "%s: %s must be a non-NULL 16-byte aligned device pointer", who, name);
    if (ld < n || ld % per)
        return fail(DSPK_EINVAL, "%s: leading dimension %lld of %s must be >= %d and a multiple of %lld", who,
                    (long long)ld, name, n, (long long)per);
    return DSPK_OK;
}

int check_codes(const void *p, int64_t ld, int32_t n, const float *scales, const char *name, const char *who) {
    if (!pointer(p, 16)) return fail(DSPK_EINVAL, "%s: %s must be a non-NULL 16-byte aligned device pointer", who, name);
    if (ld < n || ld % 16)
        return fail(DSPK_EINVAL, "%s: leading dimension %lld of %s must be >= %d and a multiple of 16", who,
                    (long long)ld, name, n);
    if (!pointer(scales, 4)) return fail(DSPK_EINVAL, "%s: the scales of %s are NULL or misaligned", who, name);
    return DSPK_OK;
}

int check_width(int32_t m, int32_t n, const char *who) {
    if (m < 0) return fail(DSPK_EINVAL, "%s: m=%d must be >= 0", who, m);
    if (n < 1) return fail(DSPK_EINVAL, "%s: n=%d must be >= 1", who, n);
    if (n > DSPK_MAX_WIDTH) return fail(DSPK_EUNSUPPORTED, "%s: n=%d (at most %d)", who, n, DSPK_MAX_WIDTH);
    return DSPK_OK;
}

// y of the products: rows [m][ldy], elements alone aligned.
int check_y(const void *y, int64_t ldy, int32_t n, const char *who) {
    if (!pointer(y, 4)) return fail(DSPK_EINVAL, "%s: y NULL or misaligned", who);
    if (ldy < n) return fail(DSPK_EINVAL, "%s: ldy=%lld < n=%d", who, (long long)ldy, n);
    return DSPK_OK;
}

int check_out(const dspk_rows_out *out, dspk::RowArgs &A, const char *who) {
    if (out->rows != nullptr) {
        int rc = check_rows(out->rows, out->ld, A.n, DSPK_BF16, "out.rows", who);
        if (rc) return rc;
    }
    if (out->codes != nullptr) {
        int rc = check_codes(out->codes, out->ldc, A.n, out->scales, "out.codes", who);
        if (rc) return rc;
    }
    A.rows = out->rows;
    A.ld = out->ld;
    A.codes = out->codes;
    A.ldc = out->ldc;
    A.scales = out->scales;
    return DSPK_OK;
}

int check_some_out(const dspk_rows_out *out, const char *who) {
    if (out == nullptr || (out->rows == nullptr && out->codes == nullptr))
        return fail(DSPK_EINVAL, "%s: out is NULL, or has neither rows nor codes", who);
    if (out->codes == nullptr && out->scales != nullptr) return fail(DSPK_EINVAL, "%s: out.scales without out.codes", who);
    return DSPK_OK;
}

int check_i8_shape(int32_t n, int32_t k, int32_t count, const char *who) {
    if (n < 1 || k < 1 || count < 1)
        return fail(DSPK_EINVAL, "%s: n=%d, k=%d and count=%d must be >= 1", who, n, k, count);
    if (k > DSPK_I8_MAX_K) return fail(DSPK_EUNSUPPORTED, "%s: k=%d (at most %d)", who, k, DSPK_I8_MAX_K);
    return DSPK_OK;
}

int check_i8_weight(const dspk_i8_weight *w, const char *name, const char *who) {
    if (w == nullptr) return fail(DSPK_EINVAL, "%s: %s is NULL", who, name);
    int rc = check_i8_shape(w->n, w->k, w->count, who);
    if (rc) return rc;
    if (!pointer(w->tiles, 256) || !pointer(w->scales, 4))
        return fail(DSPK_EINVAL, "%s: tiles of %s must be 256-byte aligned, its scales 4-byte aligned, neither NULL", who,
                    name);
    return DSPK_OK;
}

// The sizes of an expert layer; 0: fine.
int check_moe(int32_t m, int32_t experts, int32_t top_k, const char *who) {
    if (m < 0 || m > DSPK_MOE_MAX_ROWS) return fail(DSPK_EINVAL, "%s: m=%d out of 0..%d", who, m, DSPK_MOE_MAX_ROWS);
    if (experts < 1 || experts > DSPK_MOE_MAX_EXPERTS)
        return fail(DSPK_EINVAL, "%s: experts=%d out of 1..%d", who, experts, DSPK_MOE_MAX_EXPERTS);
    if (top_k < 1 || top_k > DSPK_MOE_MAX_TOP)
        return fail(DSPK_EINVAL, "%s: top_k=%d out of 1..%d", who, top_k, DSPK_MOE_MAX_TOP);
    return DSPK_OK;
}

int check_workspace(const void *ws, size_t bytes, size_t need, const char *who) {
    if (!pointer(ws, 256) || bytes < need)
        return fail(DSPK_EINVAL, "%s: workspace of %zu bytes required (256-byte aligned)", who, need);
    return DSPK_OK;
}

}  // namespace

extern "C" {

int dspk_add_rmsnorm(const void *x, int64_t ldx, int32_t x_dtype, const void *residual, int64_t ldr, int32_t r_dtype,
                     void *residual_out, int64_t ldro, const float *weight, float eps, int32_t m, int32_t n,
                     const dspk_rows_out *out, void *stream) {
    const char *who = "dspk_add_rmsnorm";
    dspk::RowArgs A{};
    int rc = check_width(m, n, who);
    if (rc || (rc = check_dtype(x_dtype, "x", who)) || (rc = check_dtype(r_dtype, "residual", who))) return rc;
    if (!(eps >= 0.f) || !isfinite(eps)) return fail(DSPK_EINVAL, "%s: eps must be finite and >= 0", who);
    if (!aligned(weight, 16)) return fail(DSPK_EINVAL, "%s: weight must be 16-byte aligned", who);
    if (m == 0) return ok();
    if ((rc = check_some_out(out, who))) return rc;
    if (x == nullptr && residual == nullptr) return fail(DSPK_EINVAL, "%s: x and residual are both NULL", who);
    A.m = m;
    A.n = n;
    if ((x != nullptr && (rc = check_rows(x, ldx, n, x_dtype, "x", who))) ||
        (residual != nullptr && (rc = check_rows(residual, ldr, n, r_dtype, "residual", who))) ||
        (residual_out != nullptr && (rc = check_rows(residual_out, ldro, n, r_dtype, "residual_out", who))) ||
        (rc = check_out(out, A, who)))
        return rc;
    if (residual_out != nullptr && ((residual_out == residual && ldro != ldr) ||
                                    (residual_out == x && (r_dtype != x_dtype || ldro != ldx))))
        return fail(DSPK_EINVAL, "%s: residual_out may be residual or x only with its type and leading dimension", who);
    A.x = x;
    A.ldx = ldx;
    A.x_f32 = x_dtype == DSPK_F32;
    A.r = residual;
    A.ldr = ldr;
    A.r_f32 = r_dtype == DSPK_F32;
    A.r_out = residual_out;
    A.ldro = ldro;
    A.w = weight;
    A.eps = eps;
    return launch_result(dspk::launch_rows(dspk::kRowNorm, A, dspk::device_cus(), (hipStream_t)stream), who);
}

int dspk_silu_mul(const void *gate, int64_t ldg, const void *up, int64_t ldu, int32_t dtype, int32_t m, int32_t n,
                  const dspk_rows_out *out, void *stream) {
    const char *who = "dspk_silu_mul";
    dspk::RowArgs A{};
    int rc = check_width(m, n, who);
    if (rc || (rc = check_dtype(dtype, "gate and up", who))) return rc;
    if (m == 0) return ok();
    if ((rc = check_some_out(out, who))) return rc;
    A.m = m;
    A.n = n;
    if ((rc = check_rows(gate, ldg, n, dtype, "gate", who)) || (rc = check_rows(up, ldu, n, dtype, "up", who)) ||
        (rc = check_out(out, A, who)))
        return rc;
    A.x = gate;
    A.ldx = ldg;
    A.r = up;
    A.ldr = ldu;
    A.x_f32 = A.r_f32 = dtype == DSPK_F32;
    return launch_result(dspk::launch_rows(dspk::kRowSilu, A, dspk::device_cus(), (hipStream_t)stream), who);
}

int dspk_i8_quantize(const void *x, int64_t ldx, int32_t dtype, int32_t m, int32_t n, int8_t *codes, int64_t ldc,
                     float *scales, void *stream) {
    const char *who = "dspk_i8_quantize";
    dspk::RowArgs A{};
    int rc = check_width(m, n, who);
    if (rc || (rc = check_dtype(dtype, "x", who))) return rc;
    if (m == 0) return ok();
    if ((rc = check_rows(x, ldx, n, dtype, "x", who)) || (rc = check_codes(codes, ldc, n, scales, "codes", who))) return rc;
    A.m = m;
    A.n = n;
    A.x = x;
    A.ldx = ldx;
    A.x_f32 = dtype == DSPK_F32;
    A.codes = codes;
    A.ldc = ldc;
    A.scales = scales;
    return launch_result(dspk::launch_rows(dspk::kRowPlain, A, dspk::device_cus(), (hipStream_t)stream), who);
}

int dspk_i8_read(const int8_t *codes, int64_t ldc, const float *scales, int32_t m, int32_t n, void *y, int64_t ldy,
                 int32_t dtype, void *stream) {
    const char *who = "dspk_i8_read";
    int rc = check_width(m, n, who);
    if (rc || (rc = check_dtype(dtype, "y", who))) return rc;
    if (m == 0) return ok();
    if ((rc = check_codes(codes, ldc, n, scales, "codes", who)) || (rc = check_rows(y, ldy, n, dtype, "y", who))) return rc;
    const dspk::I8ReadArgs A = {codes, ldc, scales, m, n, y, ldy, dtype == DSPK_F32};
    return launch_result(dspk::launch_i8_read(A, (hipStream_t)stream), who);
}

size_t dspk_i8_tiled_bytes(int32_t n, int32_t k, int32_t count) {
    if (check_i8_shape(n, k, count, "dspk_i8_tiled_bytes")) return 0;
    const size_t one = (size_t)dspk::i8_tiles(n) * dspk::i8_steps(k) * dspk::kI8Frag;      // < 2^49
    return one > (size_t)(SIZE_MAX / count) ? 0 : one * count;
}

int dspk_i8_pack(const int8_t *codes, int64_t ldc, int32_t n, int32_t k, int32_t count, void *tiles, size_t tiles_bytes,
                 void *stream) {
    const char *who = "dspk_i8_pack";
    int rc = check_i8_shape(n, k, count, who);
    if (rc) return rc;
    if (codes == nullptr || ldc < k) return fail(DSPK_EINVAL, "%s: codes NULL, or ldc=%lld < k=%d", who, (long long)ldc, k);
    const size_t need = dspk_i8_tiled_bytes(n, k, count);
    if (!pointer(tiles, 256) || need == 0 || tiles_bytes < need)
        return fail(DSPK_EINVAL, "%s: tiles of %zu bytes required (256-byte aligned)", who, need);
    const dspk::I8PackArgs A = {codes, ldc, n, k, (int32_t)dspk::i8_tiles(n), (int32_t)dspk::i8_steps(k), dspk::i8_tiles(n) * count, tiles};
    return launch_result(dspk::launch_i8_pack(A, (hipStream_t)stream), who);
}

size_t dspk_i8_workspace_bytes(int32_t n, int32_t k, int32_t m) {
    if (check_i8_shape(n, k, 1, "dspk_i8_workspace_bytes") || m < 1) return 0;
    return dspk::i8_plan(n, k, m, true, dspk::device_cus()).ws_bytes;
}

int dspk_i8_gemm(const dspk_i8_weight *w, const int8_t *x, int64_t ldx, const float *x_scales, int32_t m, void *y,
                 int32_t y_dtype, int64_t ldy, void *workspace, size_t ws_bytes, void *stream) {
    const char *who = "dspk_i8_gemm";
    int rc = check_i8_weight(w, "w", who);
    if (rc) return rc;
    if (w->count != 1) return fail(DSPK_EINVAL, "%s: a weight of count=%d (must be 1)", who, w->count);
    if (m < 0) return fail(DSPK_EINVAL, "%s: m=%d must be >= 0", who, m);
    if ((rc = check_dtype(y_dtype, "y", who))) return rc;
    if (m == 0) return ok();
    if ((rc = check_codes(x, ldx, w->k, x_scales, "x", who)) || (rc = check_y(y, ldy, w->n, who))) return rc;
    // the rows of a tile are numbered in 32 bits
    if (ldx > 1 << 24) return fail(DSPK_EUNSUPPORTED, "%s: ldx=%lld (at most 2^24)", who, (long long)ldx);
    const dspk::I8Plan p = dspk::i8_plan(w->n, w->k, m, workspace != nullptr, dspk::device_cus());
    if (!p.fits) return fail(DSPK_EUNSUPPORTED, "%s: n=%d, m=%d: too many tiles for one launch", who, w->n, m);
    if (workspace != nullptr && (rc = check_workspace(workspace, ws_bytes, p.ws_bytes, who))) return rc;
    dspk::I8GemmArgs A{};
    A.tiles = (const char *)w->tiles;
    A.w_scales = w->scales;
    A.x = x;
    A.x_scales = x_scales;
    A.y = y;
    A.ldx = ldx;
    A.ldy = ldy;
    A.m = m;
    A.n = w->n;
    A.k = w->k;
    A.tiles_n = (int32_t)dspk::i8_tiles(w->n);
    A.steps = (int32_t)dspk::i8_steps(w->k);
    A.y_bf16 = y_dtype == DSPK_BF16;
    A.vec = ldy % 4 == 0 && aligned(y, A.y_bf16 ? 8 : 16);
    A.whole = (int32_t)p.whole;
    A.splits = p.splits;
    A.ctr = (uint32_t *)workspace;
    A.part = (int32_t *)((char *)workspace + p.off_part);
    return launch_result(dspk::launch_i8_gemm(A, p, (hipStream_t)stream), who);
}

size_t dspk_moe_workspace_bytes(int32_t hidden, int32_t inter, int32_t experts, int32_t m, int32_t top_k) {
    const char *who = "dspk_moe_workspace_bytes";
    if (check_moe(m, experts, top_k, who) || m < 1 || check_i8_shape(inter, hidden, experts, who) ||
        check_i8_shape(hidden, inter, experts, who))
        return 0;
    return dspk::moe_plan(hidden, inter, experts, m, top_k, dspk::device_cus()).ws_bytes;
}

int dspk_moe_route(const uint16_t *x, int64_t ldx, const uint16_t *router, int64_t ldr, int32_t m, int32_t k,
                   int32_t experts, int32_t top_k, int32_t normalize, int32_t *ids, float *weights, float *scores,
                   int64_t lds, void *workspace, size_t ws_bytes, void *stream) {
    const char *who = "dspk_moe_route";
    int rc = check_moe(m, experts, top_k, who);
    if (rc) return rc;
    if (top_k > experts) return fail(DSPK_EINVAL, "%s: top_k=%d of %d experts", who, top_k, experts);
    if (k < 1) return fail(DSPK_EINVAL, "%s: k=%d must be >= 1", who, k);
    if (normalize != 0 && normalize != 1) return fail(DSPK_EINVAL, "%s: normalize=%d (0 or 1)", who, normalize);
    if (m == 0) return ok();
    if ((rc = check_rows(x, ldx, k, DSPK_BF16, "x", who)) || (rc = check_rows(router, ldr, k, DSPK_BF16, "router", who)))
        return rc;
    if (!pointer(ids, 4) || !pointer(weights, 4)) return fail(DSPK_EINVAL, "%s: ids or weights NULL or misaligned", who);
    if (!aligned(scores, 4) || (scores != nullptr && lds < experts))
        return fail(DSPK_EINVAL, "%s: scores misaligned, or lds=%lld < experts=%d", who, (long long)lds, experts);
    const size_t at = dspk::moe_plan(1, 1, experts, m, top_k, dspk::device_cus()).off_scores, need = at + (size_t)m * experts * sizeof(float);
    if ((rc = check_workspace(workspace, ws_bytes, need, who))) return rc;
    dspk::RouteArgs A{};
    A.x = x;
    A.ldx = ldx;
    A.router = router;
    A.ldr = ldr;
    A.m = m;
    A.k = k;
    A.experts = experts;
    A.top_k = top_k;
    A.normalize = normalize;
    A.ids = ids;
    A.weights = weights;
    A.scores = scores;
    A.lds = lds;
    A.part = (float *)((char *)workspace + at);
    A.counter = (uint32_t *)workspace;
    return launch_result(dspk::launch_moe_route(A, (hipStream_t)stream), who);
}

int dspk_moe_mlp(const dspk_i8_weight *gate, const dspk_i8_weight *up, const dspk_i8_weight *down, const int8_t *x,
                 int64_t ldx, const float *x_scales, int32_t m, const int32_t *ids, const float *weights, int32_t top_k,
                 void *y, int32_t y_dtype, int64_t ldy, void *workspace, size_t ws_bytes, void *stream) {
    const char *who = "dspk_moe_mlp";
    int rc = check_i8_weight(gate, "gate", who);
    if (rc || (rc = check_i8_weight(up, "up", who)) || (rc = check_i8_weight(down, "down", who))) return rc;
    const int32_t hidden = gate->k, inter = gate->n, experts = gate->count;
    if ((rc = check_moe(m, experts, top_k, who))) return rc;
    if (up->n != inter || up->k != hidden || up->count != experts || down->n != hidden || down->k != inter ||
        down->count != experts)
        return fail(DSPK_EINVAL, "%s: gate, up and down of different sizes", who);
    if ((rc = check_dtype(y_dtype, "y", who))) return rc;
    if (m == 0) return ok();
    if ((rc = check_codes(x, ldx, hidden, x_scales, "x", who)) || (rc = check_y(y, ldy, hidden, who))) return rc;
    if (!pointer(ids, 4) || !pointer(weights, 4)) return fail(DSPK_EINVAL, "%s: ids or weights NULL or misaligned", who);
    const dspk::MoePlan p = dspk::moe_plan(hidden, inter, experts, m, top_k, dspk::device_cus());
    if ((rc = check_workspace(workspace, ws_bytes, p.ws_bytes, who))) return rc;
    dspk::MoeArgs A{};
    A.gate = (const char *)gate->tiles;
    A.up = (const char *)up->tiles;
    A.down = (const char *)down->tiles;
    A.gate_scales = gate->scales;
    A.up_scales = up->scales;
    A.down_scales = down->scales;
    A.x = x;
    A.ldx = ldx;
    A.x_scales = x_scales;
    A.m = m;
    A.hidden = hidden;
    A.inter = inter;
    A.experts = experts;
    A.top_k = top_k;
    A.ids = ids;
    A.weights = weights;
    A.y = y;
    A.ldy = ldy;
    A.y_bf16 = y_dtype == DSPK_BF16;
    char *ws = (char *)workspace;
    A.ldh = p.ldh;
    A.h = (float *)(ws + p.off_h);
    A.h8 = (int8_t *)(ws + p.off_h8);
    A.h_scales = (float *)(ws + p.off_h_scales);
    A.ctr = (uint32_t *)(ws + dspk::kMoeCtr);
    A.top = (uint32_t *)(ws + p.off_top);
    A.parts = p.parts;
    A.inside = p.inside;
    A.part = (int32_t *)(ws + p.off_part);
    A.down_ctr = (uint32_t *)(ws + dspk::kMoeDown);
    return launch_result(dspk::launch_moe_mlp(A, (hipStream_t)stream), who);
}

}  // extern "C"
