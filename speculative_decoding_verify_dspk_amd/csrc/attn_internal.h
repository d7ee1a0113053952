// Internal declarations of the attention side of the pass (paged k/v cache,
// attention over it, tree bookkeeping), shared by its C-ABI layer and kernels.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace dspk {

constexpr int kBlockShift = 6;      // log2 of the positions per block of the cache
constexpr int kBlockTokens = 1 << kBlockShift;      // a page is 2^k blocks
constexpr int kMaxTree = 64;        // rows of one request in an attention or tree call (one mask bit each)
constexpr int kMaxCaches = 64;      // caches (layers) of one commit launch
constexpr int64_t kLaunchThreads = UINT32_MAX;      // most threads of a launch's dimension
constexpr int kManyQRows = 4;       // q rows of an append's workgroup, of many

// The paged cache; see the layout at dspk_kv_cache.
struct KvCache {
    int32_t heads, d, bits;
    int32_t page_shift;             // log2 of the positions per page
    int64_t pages;
    void *k, *v;
    float *ks, *vs;                 // 8-bit caches
};

// The requests of a call; see dspk_attn_batch.
struct AttnBatch {
    int32_t b, max_rows, total_rows, max_pages;
    const int32_t *row_start, *cache_len, *page_table;
};

// Shape of an append or read-back launch: workgroups of kRowThreads, one for each
// block of 2^bs positions that a request of the call can touch and each k/v head,
// then those of the q rows; see kv_cache.hip.
constexpr int kRowThreads = 256;
struct RowsPlan {
    int32_t bs, nb;                 // log2 of a block's positions, blocks per request
    int32_t kv_blocks;              // workgroups of the k/v rows
    int32_t q_rows, q_blocks, slices;   // rows of a q workgroup, workgroups per request, slices of a row's heads
    int32_t grid;
    bool fits;                      // the launch's threads fit 32 bits
};
RowsPlan rows_plan(const AttnBatch &B, int32_t heads, int32_t d, int32_t q_heads, bool read);

struct AppendArgs {
    KvCache c;
    AttnBatch B;
    RowsPlan g;
    const void *q, *k, *v;          // rows [total_rows][ld]; q NULL: none
    int64_t ldq, ldk, ldv;
    int32_t q_heads;
    int32_t f32;                    // rows are fp32, else bf16
    float eps;
    const float *qw, *kw;           // norm weights [d], or NULL: no norm
    const float *inv_freq;          // [rot/2], or NULL: no rotation
    int32_t rot, interleaved;
    const int32_t *positions;       // [total_rows], or NULL: cache position
    uint16_t *q_out;
    int64_t ldqo;
};
hipError_t launch_append(const AppendArgs &a, hipStream_t s);

struct ReadArgs {
    KvCache c;
    AttnBatch B;
    RowsPlan g;
    void *k, *v;                    // rows [total_rows][ld]
    int64_t ldk, ldv;
    int32_t f32;
};
hipError_t launch_kv_read(const ReadArgs &a, hipStream_t s);

struct CachePtrs {
    void *k, *v;
    float *ks, *vs;
};
struct CommitArgs {
    KvCache c;                      // geometry (its pointers are unused)
    AttnBatch B;                    // max_rows: nodes per request
    const int32_t *path, *accept_len;
    int32_t *new_len;               // or NULL
    int32_t count;
    CachePtrs caches[kMaxCaches];
};
hipError_t launch_kv_commit(const CommitArgs &a, hipStream_t s);
// new_len[r] alone, for a call whose new_len is its cache_len
hipError_t launch_new_len(const CommitArgs &a, hipStream_t s);

// Shape of an attention launch: groups of `blocks` workgroups, one per block of
// `tiles` x 16 rows; see tree_attn.hip.
constexpr int kAttnWaves = 8;
constexpr int kAttnStep = 32;                       // positions of a wave's step
constexpr int kAttnTile = 256 + 32;                 // floats of a 16 x 16 tile of partial sums, with m and sum of its rows
constexpr int kAttnCounter = 16;                   // words from one arrival counter to the next: a memory line each
constexpr int64_t kAttnJoinBytes = 64 << 10;        // partial sums of a segment's row block above which their addition gets a launch
constexpr int attn_tiles(int d) { return d == 256 ? 1 : 2; }         // most row tiles of a wave (its registers)
constexpr int attn_piece(int d, int rt) { return rt * (d / 16) * kAttnTile; }  // floats of a row block's partial sums
struct AttnPlan {
    int32_t tiles, blocks, groups;
    int32_t join;                   // shared segments are added by a launch of their own
    int32_t pairs;                  // segments are of two units at most, by the page table's width
    bool fits;                      // unit numbers fit 31 bits
    size_t off_part, ws_bytes;      // workspace: counters, then partial sums
};
AttnPlan attn_plan(int32_t q_heads, int32_t kv_heads, int32_t d, int32_t b, int32_t max_rows, int64_t capacity,
                   int cus);

struct AttnArgs {
    KvCache c;
    AttnBatch B;
    const uint16_t *q;
    uint16_t *out;
    int64_t ldq, ldo;
    int32_t rep;                    // q heads per kv head
    float scale;                    // of the scores, times log2(e)
    const uint64_t *mask;           // [total_rows], or NULL: a chain
    int32_t tiles, blocks, groups, join, pairs;      // see AttnPlan
    uint32_t *counters;             // arrivals at shared segments [groups][blocks][waves][kAttnCounter], zero between calls
    float *part;                    // partial sums [groups][blocks][2][attn_piece]
};
hipError_t launch_tree_attention(const AttnArgs &a, hipStream_t s);

hipError_t launch_tree_layout(const int32_t *parents, int32_t b, int32_t m, const int32_t *cache_len, uint64_t *mask,
                              int32_t *positions, hipStream_t s);
hipError_t launch_accept_tree(const int32_t *target, const int32_t *draft, const int32_t *parents, int32_t b, int32_t m,
                              int32_t *accept_len, int32_t *committed, int32_t *path, hipStream_t s);

// Stores the thread's error message (dspk_last_error) and returns `code`.
int set_error(int code, const char *msg);

}  // namespace dspk
