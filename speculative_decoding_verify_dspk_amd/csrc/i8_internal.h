// Internal declarations of the 8-bit integer side of a layer (row kernels,
// products of 8-bit rows with 8-bit weights, expert layers), shared by its C-ABI
// layer and kernels.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace dspk {

// ---- rows: norm, activation, quantising -------------------------------------
enum RowOp : int { kRowNorm = 0, kRowSilu = 1, kRowPlain = 2 };
struct RowArgs {
    const void *x;                  // [m][ldx]; norm: or NULL; silu: gate
    const void *r;                  // norm: residual, or NULL; silu: up
    void *r_out;                    // norm: [m][ldro] of r's type, or NULL
    int64_t ldx, ldr, ldro;
    int32_t x_f32, r_f32;           // element types: fp32, else bf16
    const float *w;                 // norm: [n], or NULL
    float eps;
    int32_t m, n;
    uint16_t *rows;                 // outputs; see dspk_rows_out
    int64_t ld;
    int8_t *codes;
    int64_t ldc;
    float *scales;
};
constexpr int kRowPiece = 8;        // columns of a lane's piece
constexpr int kRowMostThreads = 1024;
hipError_t launch_rows(RowOp op, const RowArgs &a, int cus, hipStream_t s);

struct I8ReadArgs {
    const int8_t *codes;
    int64_t ldc;
    const float *scales;
    int32_t m, n;
    void *y;
    int64_t ldy;
    int32_t y_f32;
};
hipError_t launch_i8_read(const I8ReadArgs &a, hipStream_t s);

// ---- weights and products ----------------------------------------------------
// A weight is fragments of 16 columns x 64 K, 1 KiB each, K fastest, an even number
// of them (K is filled up with zeros): lane l of a wave holds column l % 16, K
// 16 (l / 16) .. + 15, its operand of a 16x16x64 matrix instruction.
constexpr int kI8Cols = 16, kI8K = 64, kI8Frag = kI8Cols * kI8K;
constexpr int64_t i8_tiles(int64_t n) { return (n + kI8Cols - 1) / kI8Cols; }
constexpr int64_t i8_steps(int64_t k) { return (k + 2 * kI8K - 1) / (2 * kI8K) * 2; }
struct I8PackArgs {
    const int8_t *codes;
    int64_t ldc;
    int32_t n, k, tiles_n, steps;   // tiles of 16 columns of one weight, fragments of a tile
    int64_t tiles;                  // of all weights
    void *out;
};
hipError_t launch_i8_pack(const I8PackArgs &a, hipStream_t s);

struct I8GemmArgs {
    const char *tiles;
    const float *w_scales;
    const int8_t *x;
    const float *x_scales;
    void *y;
    int64_t ldx, ldy;
    int32_t m, n, k;
    int32_t tiles_n, steps;         // tiles of 16 columns, fragments of a tile
    int32_t y_bf16;
    int32_t vec;                    // four neighbouring columns of y are stored at once
    int32_t whole;                  // 256 x 256 tiles that are not cut into four
    int32_t splits;                 // of K; > 1 needs the two regions below
    int32_t *part;                  // sums [tile][split][wave][..]
    uint32_t *ctr;                  // arrivals [tile], zero between calls
};
// Shape of a launch; see i8_gemm.hip.  Stream: rows x 16-column tiles of a workgroup;
// tile: rows x columns.
enum I8Kind : int {
    kI8Stream16x1, kI8Stream16x2, kI8Stream32x1, kI8Stream32x2, kI8Stream64x1, kI8Stream64x2,
    kI8Tile32x64, kI8Tile64x64, kI8Tile64x128, kI8Tile128x128, kI8Tile256x256
};
struct I8Plan {
    I8Kind kind;
    int32_t waves;                  // stream: of a workgroup
    int32_t splits;                 // tile: of K
    int64_t whole, groups;          // 256 x 256 tiles that are not cut, workgroups
    bool fits;
    size_t off_part, ws_bytes;      // workspace: arrivals, then from kMoeHead on sums
};
constexpr int kI8MaxSplitTiles = 1024;
I8Plan i8_plan(int32_t n, int32_t k, int32_t m, bool split, int cus);
hipError_t launch_i8_gemm(const I8GemmArgs &a, const I8Plan &p, hipStream_t s);

// ---- expert layers -----------------------------------------------------------
constexpr int kMoeMaxRows = 64, kMoeMaxExperts = 1024, kMoeMaxTop = 32;
constexpr int kMoeMaxSlots = kMoeMaxRows * kMoeMaxTop;
// Workspace: what has to be zero between calls lies at fixed places below kMoeHead, the
// products' arrivals too, so that calls of any sizes and of both families share one buffer:
//   [0, 256)   arrivals of the router's workgroups
//   kMoeCtr    arrivals of each expert's columns
//   kMoeDown   arrivals at each 16 columns of y
// then the router's scores, h, its codes and their scales, and the largest magnitude of
// each row's tiles, the down workgroups' sums, each written before it is read.
constexpr int kMoeGroup = 512;      // slots that a down workgroup has sums for at a time
constexpr int kDownWaves = 16;      // of a down workgroup
constexpr int kMoeInside = 2048;    // longest row of h whose codes are made inside the down workgroups
constexpr int kMoeMaxParts = 8, kMoeSplitTiles = 512;      // tiles of 16 columns whose sums are split
constexpr size_t kMoeCtr = 256, kMoeDown = kMoeCtr + 4 * kMoeMaxExperts, kMoeHead = kMoeDown + 4 * kMoeSplitTiles;
static_assert(4 * kI8MaxSplitTiles <= kMoeHead && kMoeHead % 256 == 0, "the products' sums lie behind all arrivals");
struct MoePlan {
    int64_t ldh;                    // floats of a row of h, bytes of a row of its codes
    int32_t parts;                  // workgroups that share 16 columns of y
    bool inside;                    // h becomes codes in the down workgroups
    size_t off_scores, off_h, off_h8, off_h_scales, off_top, off_part, ws_bytes;
};
MoePlan moe_plan(int32_t hidden, int32_t inter, int32_t experts, int32_t m, int32_t top_k, int cus);

struct RouteArgs {
    const uint16_t *x, *router;
    int64_t ldx, ldr, lds;
    int32_t m, k, experts, top_k, normalize;
    int32_t *ids;
    float *weights, *scores;        // scores: or NULL
    float *part;                    // [m][experts] in the workspace
    uint32_t *counter;
};
hipError_t launch_moe_route(const RouteArgs &a, hipStream_t s);

struct MoeArgs {
    const char *gate, *up, *down;
    const float *gate_scales, *up_scales, *down_scales;
    const int8_t *x;
    const float *x_scales;
    int64_t ldx, ldy, ldh;
    int32_t m, hidden, inter, experts, top_k;
    const int32_t *ids;
    const float *weights;
    void *y;
    int32_t y_bf16;
    float *h;                       // [m * top_k][ldh]
    int8_t *h8;                     // [m * top_k][ldh], with h_scales [m * top_k]
    float *h_scales;
    uint32_t *ctr;                  // arrivals of each expert's columns
    uint32_t *top;                  // [m * top_k][tiles of 16 columns]: largest |h|, as bits
    int32_t parts, inside;          // see MoePlan
    int32_t *part;                  // their sums [tile][part][slot][16]
    uint32_t *down_ctr;             // their arrivals
};
hipError_t launch_moe_mlp(const MoeArgs &a, hipStream_t s);

int device_cus();
// Stores the thread's error message (dspk_last_error) and returns `code`.
int set_error(int code, const char *msg);

}  // namespace dspk
