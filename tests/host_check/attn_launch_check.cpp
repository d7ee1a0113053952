// Host-only check of the launch shapes of the cache and tree calls, built with
// AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_attn_launch_bounds.py.
//
// It links attn_api.cpp with recorders in place of the kernel launches, which
// check that a launch covers the rows of every request wherever they start, and
// that its threads fit the 32 bits a launch has.  No pointer is dereferenced.
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>
#include <string>

#include <hip/hip_runtime_api.h>

#include "attn_internal.h"
#include "dspk.h"
#include "dspk_internal.h"

static int g_fail = 0, g_launches = 0;
static std::string g_msg;
#define CHECK(c)                                                                   \
    do {                                                                           \
        if (!(c)) {                                                                \
            fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #c); \
            ++g_fail;                                                              \
        }                                                                          \
    } while (0)

extern "C" const char *hipGetErrorString(hipError_t) { return "error"; }

namespace dspk {
int set_error(int code, const char *msg) {
    g_msg = msg;
    return code;
}
int device_cus() { return 256; }

static void check_rows_plan(const RowsPlan &g, const AttnBatch &B, int32_t heads, int32_t d, int32_t q_heads) {
    const int64_t rows = B.max_rows < B.total_rows ? B.max_rows : B.total_rows, block = 1ll << g.bs;
    CHECK(g.bs == kBlockShift || g.bs == kBlockShift - 1);
    for (int64_t start : {0, 1, 31, 32, 62, 63})                      // positions rows start..  lie in blocks 0 .. nb - 1
        if (rows > 0) CHECK((start % block + rows - 1) / block < g.nb);
    CHECK((int64_t)g.nb * B.b * heads == g.kv_blocks);
    int64_t q = 0;
    if (q_heads > 0) {
        CHECK(g.q_rows >= 1 && g.q_rows <= kManyQRows && (int64_t)g.q_rows * g.q_blocks >= rows);
        CHECK(g.slices >= 1 && (int64_t)(g.slices - 1) * 2048 < (int64_t)q_heads * d);
        q = (int64_t)B.b * g.q_blocks * g.slices;
    }
    CHECK(g.grid == g.kv_blocks + q && (int64_t)g.grid * kRowThreads <= UINT32_MAX);
    // the last block's positions stay within 31 bits, from any length up to 2^30
    CHECK((((1ll << 30 >> g.bs) + g.nb - 1) << g.bs) + block <= 1ll << 31);
}
hipError_t launch_append(const AppendArgs &a, hipStream_t) {
    check_rows_plan(a.g, a.B, a.c.heads, a.c.d, a.q == nullptr ? 0 : a.q_heads);
    return ++g_launches, hipSuccess;
}
hipError_t launch_kv_read(const ReadArgs &a, hipStream_t) {
    check_rows_plan(a.g, a.B, a.c.heads, a.c.d, 0);
    CHECK(a.g.bs == kBlockShift);
    return ++g_launches, hipSuccess;
}
hipError_t launch_kv_commit(const CommitArgs &, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_new_len(const CommitArgs &, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_tree_attention(const AttnArgs &, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_tree_layout(const int32_t *, int32_t b, int32_t, const int32_t *, uint64_t *, int32_t *, hipStream_t) {
    CHECK((int64_t)b * 64 <= UINT32_MAX);
    return ++g_launches, hipSuccess;
}
hipError_t launch_accept_tree(const int32_t *, const int32_t *, const int32_t *, int32_t b, int32_t, int32_t *, int32_t *,
                              int32_t *, hipStream_t) {
    CHECK((int64_t)b * 64 <= UINT32_MAX);
    return ++g_launches, hipSuccess;
}
}  // namespace dspk

static char *const P = (char *)0x10000000;
static int32_t *const I = (int32_t *)P;

// The three row calls with one batch; each launches, or refuses without a launch.
static int calls(const dspk_kv_cache &c, const dspk_attn_batch &B, int32_t hq, int rc[3]) {
    const dspk_qk_prep prep = {1e-6f, nullptr, nullptr, nullptr, 0, 0, nullptr};
    const int64_t ld = (int64_t)c.kv_heads * c.head_dim, ldq = (int64_t)hq * c.head_dim;
    int n = 0;
    for (int i = 0; i < 3; ++i) {
        const int before = g_launches;
        rc[i] = i == 0 ? dspk_kv_append(&c, &B, P, ld, P, ld, DSPK_BF16, nullptr)
              : i == 1 ? dspk_kv_read(&c, &B, P, ld, P, ld, DSPK_BF16, nullptr)
                       : dspk_qkv_norm_rope_append(&c, &B, &prep, P, ldq, P, ld, P, ld, DSPK_BF16, hq, (uint16_t *)(P + 4096),
                                                   ldq, nullptr);
        CHECK(rc[i] == DSPK_OK || rc[i] == DSPK_EUNSUPPORTED);
        CHECK(g_launches == before + (rc[i] == DSPK_OK));
        n += rc[i] == DSPK_OK;
    }
    return n;
}

int main() {
    int rc[3];
    for (int hkv : {1, 8, 65535})
        for (int d : {64, 256})
            for (int hq : {1, 32, 65535})
                for (int b : {1, 3, 512, 65535})
                    for (int64_t rows : {1ll, 2ll, 63ll, 64ll, 65ll, 100000ll, (1ll << 24) - 1, 1ll << 24, 1ll << 30, (1ll << 31) - 1})
                        for (int64_t total : {0ll, 1ll, 1000ll, 110000ll, (1ll << 30) + 1, (1ll << 31) - 1}) {
                            const dspk_kv_cache c = {hkv, d, 64, 16, 1 << 20, P, P, nullptr, nullptr};
                            const dspk_attn_batch B = {b, (int32_t)rows, (int32_t)total, 9, I, I, I};
                            const int n = calls(c, B, hq, rc);
                            if (b == 1 && hkv <= 8 && hq <= 32 && (total <= 110000 || rows <= 100000)) CHECK(n == 3);
                        }
    // one request, one head: 2^24 - 1 workgroups of 64 positions, and not one more
    const dspk_kv_cache c = {1, 64, 64, 16, 1 << 20, P, P, nullptr, nullptr};
    dspk_attn_batch B = {1, (1 << 30) - 2 * 64 + 1, 2147483647, 9, I, I, I};
    calls(c, B, 1, rc);
    CHECK(rc[0] == DSPK_OK && rc[1] == DSPK_OK && rc[2] == DSPK_EUNSUPPORTED);
    ++B.max_rows;
    calls(c, B, 1, rc);
    CHECK(rc[0] == DSPK_EUNSUPPORTED && rc[1] == DSPK_EUNSUPPORTED && g_msg.find("too many rows") != std::string::npos);
    // rows that the arrays do not hold are not counted
    B.total_rows = 5000;
    CHECK(calls(c, B, 1, rc) == 3);
    // Attention: a call that is accepted, and calls that differ from it in one thing
    const dspk_kv_cache kv = {8, 128, 64, 16, 100, P, P, nullptr, nullptr};
    const dspk_attn_batch two = {2, 4, 8, 9, nullptr, I, I};
    const size_t need = dspk_attn_workspace_bytes(32, 8, 128, 2, 4);
    const auto attend = [&](int64_t ldq, int32_t hq, float scale, char *mask, char *out, int64_t ldo, char *ws, size_t bytes) {
        return dspk_tree_attention(&kv, &two, (uint16_t *)P, ldq, hq, scale, (uint64_t *)mask, (uint16_t *)out, ldo, ws, bytes,
                                   nullptr);
    };
    char *const out = P + (1 << 20), *const ws = P + (1 << 24);
    int before = g_launches;
    CHECK(attend(4096, 32, 0.1f, nullptr, out, 4096, ws, need) == DSPK_OK && g_launches == before + 1);
    CHECK(attend(4096, 32, 0.1f, P + 8, out, 4096, ws, need) == DSPK_OK && g_launches == before + 2);
    before = g_launches;
    const auto refused = [&](int rc, const char *text) {
        CHECK(rc == DSPK_EINVAL && g_launches == before && g_msg.find(text) != std::string::npos);
    };
    refused(attend(4090, 32, 0.1f, nullptr, out, 4096, ws, need), "of q");
    refused(attend(4096, 12, 0.1f, nullptr, out, 4096, ws, need), "q_heads=12");
    refused(attend(4096, 32, 0.f, nullptr, out, 4096, ws, need), "scale");
    refused(attend(4096, 32, 0.1f, P + 4, out, 4096, ws, need), "tree_mask");
    refused(attend(4096, 32, 0.1f, nullptr, P, 4096, ws, need), "out must not be q");
    refused(attend(4096, 32, 0.1f, nullptr, out, 4088, ws, need), "of out");
    refused(attend(4096, 32, 0.1f, nullptr, out, 4096, nullptr, need), "workspace");
    refused(attend(4096, 32, 0.1f, nullptr, out, 4096, ws + 128, need), "workspace");
    refused(attend(4096, 32, 0.1f, nullptr, out, 4096, ws, need - 1), "workspace");
    // requests of a tree call
    int32_t *const X = (int32_t *)(P + (1 << 20));
    CHECK(dspk_tree_layout(I, (1 << 26) - 1, 4, X, (uint64_t *)P, X, nullptr) == DSPK_OK);
    CHECK(dspk_tree_layout(I, 1 << 26, 4, X, (uint64_t *)P, X, nullptr) == DSPK_EUNSUPPORTED);
    CHECK(dspk_accept_tree_greedy(I, I, I, (1 << 26) - 1, 4, X, X, X, nullptr) == DSPK_OK);
    CHECK(dspk_accept_tree_greedy(I, I, I, 1 << 26, 4, X, X, X, nullptr) == DSPK_EUNSUPPORTED);
    if (g_fail == 0) printf("launch check ok (%d launches)\n", g_launches);
    return g_fail != 0;
}
