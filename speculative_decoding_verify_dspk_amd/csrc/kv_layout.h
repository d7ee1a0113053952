// Device-side helpers of the paged cache: where an entry lies, which rows and
// positions a request has.
#pragma once

#include <hip/hip_runtime.h>

#include "attn_internal.h"

namespace dspk {
namespace kv {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// A (page, head) chunk is made of 1 KiB slots of 64 x 16 bytes, each 16-byte
// piece what one lane of a wave feeds to the matrix cores.  W elements per
// piece: 8 (bf16) or 16 (8-bit).
//   k slot: 16 positions x 4W dimensions; lane g * 16 + (t % 16) holds
//     dimensions g * W .. of its position;
//   v slot: 4W positions x 16 dimensions; lane g * 16 + (d % 16) holds, of its
//     dimension, positions jj * 16 + g * 4 + i for jj < W / 4, i < 4 -- the
//     positions whose scores the same lane holds when scores come out of
//     the matrix cores, so probabilities feed the second product in place.
template <int D, int W>
__device__ __forceinline__ uint32_t k_piece(uint32_t t, uint32_t d) {     // first element of the piece of (t, d)
    return (((t / 16) * (D / (4 * W)) + d / (4 * W)) * 64 + (d % (4 * W)) / W * 16 + t % 16) * W;
}
template <int D, int W>
__device__ __forceinline__ uint32_t v_elem(uint32_t t, uint32_t d) {      // element (t, d)
    return (((t / (4 * W)) * (D / 16) + d / 16) * 64 + (t % 16) / 4 * 16 + d % 16) * W + (t % (4 * W)) / 16 * 4 + t % 4;
}

// Rows and cached positions of request r.  Row ranges that do not fit the
// call hold no rows; a length that does not fit the page table is a fault.
struct Req {
    int32_t row0, rows;   // first row, rows
    int32_t len;          // positions cached before the rows
    bool ok;              // len and len + rows lie within the page table
};
__device__ __forceinline__ Req request(const AttnBatch &B, int page_shift, int r) {
    Req q;
    if (B.row_start != nullptr) {
        const int64_t a = B.row_start[r], e = B.row_start[r + 1];
        const bool in = a >= 0 && e >= a && e - a <= B.max_rows && e <= B.total_rows;
        q.row0 = in ? (int32_t)a : 0;
        q.rows = in ? (int32_t)(e - a) : 0;
    } else {
        q.row0 = r * B.max_rows;
        q.rows = B.max_rows;
    }
    q.len = B.cache_len[r];
    q.ok = q.len >= 0 && (int64_t)q.len + q.rows <= ((int64_t)B.max_pages << page_shift);
    return q;
}

__device__ __forceinline__ float bf16_f32(uint32_t lo16) { return __uint_as_float(lo16 << 16); }

}  // namespace kv
}  // namespace dspk
