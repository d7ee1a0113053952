// Host-only check of the 8-bit side's C ABI, built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_i8_host_sanitize.py.
//
// It links i8_api.cpp with recorders in place of the kernel launches; every pointer is
// a made-up aligned address that nothing dereferences.  For each accepted call the
// recorders check that the launch covers the call's rows and columns, that its shape
// fits, and that what the kernels would touch of the workspace lies inside it.
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>
#include <string>

#include <hip/hip_runtime_api.h>

#include "dspk.h"
#include "i8_internal.h"

static int g_fail = 0, g_launches = 0, g_cus = 256;
static std::string g_msg;
#define CHECK(c)                                                                   \
    do {                                                                           \
        if (!(c)) {                                                                \
            fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #c); \
            ++g_fail;                                                              \
        }                                                                          \
    } while (0)

extern "C" const char *hipGetErrorString(hipError_t) { return "error"; }

static uintptr_t g_ws = 0x7000000000;
static size_t g_ws_bytes;

namespace dspk {
int set_error(int code, const char *msg) {
    g_msg = msg;
    return code;
}
int device_cus() { return g_cus; }
hipError_t launch_rows(RowOp, const RowArgs &a, int cus, hipStream_t) {
    CHECK(a.m > 0 && a.n > 0 && a.n <= DSPK_MAX_WIDTH && cus == g_cus);
    return ++g_launches, hipSuccess;
}
hipError_t launch_i8_read(const I8ReadArgs &, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_i8_pack(const I8PackArgs &a, hipStream_t) {
    CHECK(a.tiles * a.steps * kI8Frag == (int64_t)dspk_i8_tiled_bytes(a.n, a.k, (int32_t)(a.tiles / a.tiles_n)));
    CHECK(a.steps % 2 == 0 && (int64_t)a.steps * kI8K >= a.k && (int64_t)a.tiles_n * kI8Cols >= a.n);
    return ++g_launches, hipSuccess;
}
hipError_t launch_i8_gemm(const I8GemmArgs &a, const I8Plan &p, hipStream_t) {
    static const int shape[][2] = {{16, 16}, {16, 32}, {32, 16}, {32, 32}, {64, 16}, {64, 32},
                                   {32, 64}, {64, 64}, {64, 128}, {128, 128}, {256, 256}};
    const int64_t rows = shape[p.kind][0], cols = shape[p.kind][1];
    const int64_t rt = (a.m + rows - 1) / rows, ct = ((int64_t)a.n + cols - 1) / cols;
    CHECK(p.fits && p.groups >= 1);
    if (p.kind <= kI8Stream64x2) {
        CHECK(rt == 1 && p.groups == ct && p.waves >= 4 && p.waves <= 8 && p.splits == 1);
        CHECK(p.groups * 64 * p.waves <= UINT32_MAX);
        CHECK(p.waves * (rows / 16) * (cols / 16) * 1024 <= 65536);           // the waves' sums in LDS
    } else if (p.kind == kI8Tile256x256) {
        CHECK(p.splits == 1 && p.whole <= rt * ct && p.groups == p.whole + 4 * (rt * ct - p.whole));
    } else {
        CHECK(p.groups == rt * ct && p.splits >= 1);
    }
    CHECK(p.groups * 512 <= UINT32_MAX && rt * ct <= INT32_MAX);
    CHECK(a.splits == p.splits && a.whole == p.whole);
    if (p.splits > 1) {
        CHECK(p.groups <= kI8MaxSplitTiles && (a.steps / 2) / p.splits >= 4);
        const uintptr_t ctr = (uintptr_t)a.ctr + p.groups * 4;
        CHECK((uintptr_t)a.ctr == g_ws && ctr <= (uintptr_t)a.part);
        CHECK((uintptr_t)a.part + p.groups * p.splits * rows * cols * 4 <= g_ws + g_ws_bytes);
    }
    // a tile's rows are numbered in 32 bits
    CHECK((rows - 1) * a.ldx + DSPK_I8_MAX_K + 256 <= UINT32_MAX);
    return ++g_launches, hipSuccess;
}
hipError_t launch_moe_route(const RouteArgs &a, hipStream_t) {
    CHECK((uintptr_t)a.counter == g_ws && (uintptr_t)a.part >= g_ws + kMoeHead);
    CHECK((uintptr_t)a.part + (size_t)a.m * a.experts * 4 <= g_ws + g_ws_bytes);
    CHECK(a.m >= 1 && a.m <= kMoeMaxRows && a.experts <= kMoeMaxExperts && a.top_k <= kMoeMaxTop);
    return ++g_launches, hipSuccess;
}
hipError_t launch_moe_mlp(const MoeArgs &a, hipStream_t) {
    const size_t slots = (size_t)a.m * a.top_k, tiles = (a.inter + 15) / 16, cols = (a.hidden + 15) / 16;
    CHECK(a.ldh % 16 == 0 && a.ldh >= a.inter && slots <= kMoeMaxSlots);
    CHECK((uintptr_t)a.ctr >= g_ws + 256 && (uintptr_t)a.ctr + 4 * kMoeMaxExperts <= (uintptr_t)a.down_ctr);
    CHECK((uintptr_t)a.down_ctr + 4 * kMoeSplitTiles <= g_ws + kMoeHead && (uintptr_t)a.h >= g_ws + kMoeHead);
    CHECK((uintptr_t)a.h + slots * a.ldh * 4 <= (uintptr_t)a.h8);
    CHECK((uintptr_t)a.h8 + slots * a.ldh <= (uintptr_t)a.h_scales);
    CHECK((uintptr_t)a.h_scales + slots * 4 <= (uintptr_t)a.top);
    CHECK((uintptr_t)a.top + slots * tiles * 4 <= (uintptr_t)a.part);
    CHECK((uintptr_t)a.h8 % 16 == 0 && (uintptr_t)a.part % 8 == 0 && (uintptr_t)a.h % 16 == 0);
    CHECK((uintptr_t)a.part <= g_ws + g_ws_bytes);
    CHECK(a.parts >= 1 && a.parts <= kMoeMaxParts);
    if (a.parts > 1) {
        CHECK(slots <= kMoeGroup && cols <= kMoeSplitTiles);
        CHECK((uintptr_t)a.part + cols * a.parts * slots * 16 * 4 <= g_ws + g_ws_bytes);
    }
    return ++g_launches, hipSuccess;
}
}  // namespace dspk

int main() {
    char *const P = (char *)0x10000000;
    int calls = 0;
    for (int cus : {256, 304, 64, 1}) {
        g_cus = cus;
        for (int32_t n : {1, 15, 16, 17, 64, 1000, 2560, 4096, 5120, 19456, 100000, 2147483647})
            for (int32_t k : {1, 64, 65, 128, 129, 777, 2560, 9728, 17408, 131071})
                for (int32_t m : {1, 2, 16, 17, 24, 25, 32, 33, 48, 49, 64, 65, 100, 128, 129, 256, 300, 512, 1000, 4096, 30000,
                                  2147483647}) {
                    const dspk_i8_weight w = {n, k, 1, P, (float *)P};
                    const int64_t ldx = (k + 15) / 16 * 16;
                    g_ws_bytes = dspk_i8_workspace_bytes(n, k, m);
                    for (void *ws : {(void *)nullptr, (void *)g_ws}) {
                        const int before = g_launches;
                        const int rc = dspk_i8_gemm(&w, (int8_t *)P, m % 3 == 0 ? 1 << 24 : ldx, (float *)P, m, P, m % 2, n, ws,
                                                    ws == nullptr ? 0 : g_ws_bytes, nullptr);
                        ++calls;
                        CHECK(rc == DSPK_OK || (rc == DSPK_EUNSUPPORTED && g_launches == before));
                        // what fits is refused only where there are millions of tiles
                        if (rc != DSPK_OK) CHECK(((double)m / 256 + 1) * ((double)n / 16 + 1) > 4e6);
                        if (rc == DSPK_OK && g_ws_bytes && ws != nullptr)
                            CHECK(dspk_i8_gemm(&w, (int8_t *)P, ldx, (float *)P, m, P, 0, n, ws, g_ws_bytes - 1, nullptr) ==
                                  DSPK_EINVAL);
                    }
                }
        for (int32_t hidden : {1, 16, 100, 2048, 4096, 8192, 131071})
            for (int32_t inter : {1, 17, 768, 14336, 131071})
                for (int32_t experts : {1, 7, 8, 128, 1024})
                    for (int32_t m : {1, 2, 6, 16, 17, 63, 64})
                        for (int32_t top : {1, 2, 8, 32}) {
                            const dspk_i8_weight up = {inter, hidden, experts, P, (float *)P};
                            const dspk_i8_weight down = {hidden, inter, experts, P, (float *)P};
                            g_ws_bytes = dspk_moe_workspace_bytes(hidden, inter, experts, m, top);
                            CHECK(g_ws_bytes > 0);
                            const int64_t ldx = (hidden + 15) / 16 * 16;
                            CHECK(dspk_moe_mlp(&up, &up, &down, (int8_t *)P, ldx, (float *)P, m, (int32_t *)P, (float *)P, top, P,
                                               0, hidden, (void *)g_ws, g_ws_bytes, nullptr) == DSPK_OK);
                            CHECK(dspk_moe_mlp(&up, &up, &down, (int8_t *)P, ldx, (float *)P, m, (int32_t *)P, (float *)P, top, P,
                                               0, hidden, (void *)g_ws, g_ws_bytes - 1, nullptr) == DSPK_EINVAL);
                            const int rc =
                                dspk_moe_route((uint16_t *)P, ldx, (uint16_t *)P, ldx, m, hidden, experts, top, 1, (int32_t *)P,
                                               (float *)P, nullptr, 0, (void *)g_ws, g_ws_bytes, nullptr);
                            CHECK(rc == (top <= experts ? DSPK_OK : DSPK_EINVAL));
                            calls += 3;
                        }
    }
    for (int32_t n : {1, 31, 32768})
        for (int32_t m : {1, 2147483647}) {
            const int64_t ld = (n + 15) / 16 * 16;
            const dspk_rows_out out = {(uint16_t *)P, ld, (int8_t *)P, ld, (float *)P};
            CHECK(dspk_add_rmsnorm(P, ld, 1, P, ld, 0, nullptr, 0, nullptr, 0.f, m, n, &out, nullptr) == DSPK_OK);
            CHECK(dspk_silu_mul(P, ld, P, ld, 0, m, n, &out, nullptr) == DSPK_OK);
            CHECK(dspk_i8_quantize(P, ld, 0, m, n, (int8_t *)P, ld, (float *)P, nullptr) == DSPK_OK);
            CHECK(dspk_i8_read((int8_t *)P, ld, (float *)P, m, n, P, ld, 1, nullptr) == DSPK_OK);
            calls += 4;
        }
    for (int32_t count : {1, 3, 1 << 20})
        for (int32_t n : {1, 1000, 1 << 20}) {
            const size_t need = dspk_i8_tiled_bytes(n, 777, count);
            CHECK(dspk_i8_pack((int8_t *)P, 777, n, 777, count, P, need, nullptr) == DSPK_OK);
        }
    printf("%s: %d calls, %d launches\n", g_fail ? "FAILED" : "host check ok", calls, g_launches);
    return g_fail != 0;
}
