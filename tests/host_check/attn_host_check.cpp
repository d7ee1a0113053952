// Host-only check of the attention side's C ABI, built with AddressSanitizer
// and UndefinedBehaviorSanitizer by tests/test_attn_host_sanitize.py.
//
// It links attn_api.cpp with recorders in place of the kernel launches; every
// pointer is a made-up aligned address that nothing dereferences.  For each
// accepted attention call the recorder checks that what the kernels would touch
// of the workspace lies inside it, over heads, rows, lengths and CU counts.
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>
#include <string>

#include <hip/hip_runtime_api.h>

#include "attn_internal.h"
#include "dspk.h"
#include "dspk_internal.h"

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

static uintptr_t g_ws;
static size_t g_ws_bytes;

namespace dspk {
int set_error(int code, const char *msg) {
    g_msg = msg;
    return code;
}
int device_cus() { return g_cus; }
hipError_t launch_append(const AppendArgs &, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_kv_read(const ReadArgs &, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_kv_commit(const CommitArgs &a, hipStream_t) {
    CHECK(a.count >= 1 && a.count <= kMaxCaches);
    for (int i = 0; i < a.count; ++i) CHECK(a.caches[i].k != nullptr);
    return ++g_launches, hipSuccess;
}
hipError_t launch_new_len(const CommitArgs &a, hipStream_t) {
    CHECK(a.new_len == a.B.cache_len);
    return ++g_launches, hipSuccess;
}
hipError_t launch_tree_layout(const int32_t *, int32_t, int32_t, const int32_t *, uint64_t *, int32_t *, hipStream_t) {
    return ++g_launches, hipSuccess;
}
hipError_t launch_accept_tree(const int32_t *, const int32_t *, const int32_t *, int32_t, int32_t, int32_t *, int32_t *,
                              int32_t *, hipStream_t) {
    return ++g_launches, hipSuccess;
}
hipError_t launch_tree_attention(const AttnArgs &a, hipStream_t) {
    const int64_t wgs = (int64_t)a.groups * a.blocks, rows = (int64_t)a.B.max_rows * a.rep;
    CHECK(a.tiles >= 1 && a.tiles <= attn_tiles(a.c.d) && a.groups >= 1);
    CHECK((int64_t)a.blocks * a.tiles * 16 >= rows && (int64_t)(a.blocks - 1) * a.tiles * 16 < rows);
    CHECK(wgs <= (g_cus > a.blocks ? g_cus : a.blocks));              // one workgroup per CU, or one group
    const uintptr_t ctr_end = (uintptr_t)a.counters + wgs * kAttnWaves * kAttnCounter * 4;
    const uintptr_t part_end = (uintptr_t)a.part + wgs * 2 * attn_piece(a.c.d, a.tiles) * 4;
    CHECK((uintptr_t)a.counters == g_ws && ctr_end <= (uintptr_t)a.part && part_end <= g_ws + g_ws_bytes);
    // a single unit per segment leaves nothing to add
    const int64_t units = (((int64_t)a.B.max_pages << a.c.page_shift) + kAttnStep * kAttnWaves - 1) / (kAttnStep * kAttnWaves);
    if (units == 1 && a.tiles == 1 && a.c.d <= 128) CHECK(!a.join);
    return ++g_launches, hipSuccess;
}
}  // namespace dspk

int main() {
    char *const P = (char *)0x10000000;
    int32_t *const I = (int32_t *)P;
    g_ws = 0x7000000000;
    for (int cus : {256, 64, 8, 1}) {
        g_cus = cus;
        for (int d : {64, 128, 256})
            for (int hkv : {1, 2, 8})
                for (int rep : {1, 4, 5, 7, 256})
                    for (int m : {1, 2, 6, 17, 33, 64})
                        for (int b : {1, 3, 40, 300})
                            for (int pages : {1, 4, 100, 2000}) {
                                for (int bits : {8, 16}) {
                                    dspk_kv_cache c = {hkv, d, 64, bits, 1 << 20, P, P, bits == 8 ? (float *)P : nullptr,
                                                       bits == 8 ? (float *)P : nullptr};
                                    dspk_attn_batch B = {b, m, b * m, pages, nullptr, I, I};
                                    // the workspace asked for at the most rows serves fewer
                                    g_ws_bytes = dspk_attn_workspace_bytes(hkv * rep, hkv, d, b, m);
                                    CHECK(g_ws_bytes > 0 && g_ws_bytes <= dspk_attn_workspace_bytes(hkv * rep, hkv, d, b, 64));
                                    const int before = g_launches;
                                    const int64_t ld = (int64_t)hkv * rep * d;
                                    int rc = dspk_tree_attention(&c, &B, (uint16_t *)P, ld, hkv * rep, 0.1f, nullptr,
                                                                 (uint16_t *)(P + 4096), ld, (void *)g_ws, g_ws_bytes, nullptr);
                                    CHECK(rc == DSPK_OK && g_launches == before + 1);
                                    rc = dspk_tree_attention(&c, &B, (uint16_t *)P, ld, hkv * rep, 0.1f, nullptr,
                                                             (uint16_t *)(P + 4096), ld, (void *)g_ws, g_ws_bytes - 256, nullptr);
                                    CHECK(rc == DSPK_EINVAL && g_launches == before + 1 && !g_msg.empty());
                                }
                            }
    }
    // the largest sizes: no overflow on the way to a refusal
    g_cus = 256;
    dspk_kv_cache c = {65535, 256, 65536, 16, 2147483647, P, P, nullptr, nullptr};
    CHECK(dspk_kv_cache_bytes(2147483647, 65535, 256, 65536, 16) == (size_t)2147483647 * 65535 * 256 * 65536 * 2 ||
          dspk_kv_cache_bytes(2147483647, 65535, 256, 65536, 16) == 0);
    dspk_attn_batch B = {65535, 2147483647, 2147483647, 2147483647, I, I, I};
    dspk_qk_prep prep = {1e-6f, nullptr, nullptr, nullptr, 0, 0, nullptr};
    CHECK(dspk_kv_append(&c, &B, P, (int64_t)65535 * 256, P, (int64_t)65535 * 256, DSPK_BF16, nullptr) == DSPK_EUNSUPPORTED);
    CHECK(dspk_kv_read(&c, &B, P, (int64_t)65535 * 256, P, (int64_t)65535 * 256, DSPK_BF16, nullptr) == DSPK_EUNSUPPORTED);
    CHECK(dspk_qkv_norm_rope_append(&c, &B, &prep, P, (int64_t)65535 * 256, P, (int64_t)65535 * 256, P, (int64_t)65535 * 256,
                                    DSPK_BF16, 65535, (uint16_t *)P, (int64_t)65535 * 256, nullptr) == DSPK_EUNSUPPORTED);
    B.max_rows = 64;
    CHECK(dspk_tree_attention(&c, &B, (uint16_t *)P, (int64_t)65535 * 256, 65535, 1.f, nullptr, (uint16_t *)P,
                              (int64_t)65535 * 256, (void *)g_ws, (size_t)1 << 60, nullptr) == DSPK_EUNSUPPORTED);
    // commits of more caches than one launch takes
    static dspk_kv_cache many[150];
    for (auto &x : many) x = {8, 128, 64, 16, 100, P, P, nullptr, nullptr};
    dspk_attn_batch T = {4, 16, 64, 9, nullptr, I, I};
    int before = g_launches;
    CHECK(dspk_kv_commit(150, many, &T, I + 100000, I + 200000, I + 300000, nullptr) == DSPK_OK && g_launches == before + 3);
    before = g_launches;
    CHECK(dspk_kv_commit(65, many, &T, I + 100000, I + 200000, I, nullptr) == DSPK_OK && g_launches == before + 3);
    if (g_fail == 0) printf("host check ok (%d launches)\n", g_launches);
    return g_fail != 0;
}
