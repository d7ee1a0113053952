// Products of 8-bit rows with 8-bit weights, and the weights' packing:
//   y[i][c] = float(sum_r x[i][r] w[c][r]) * x_scales[i] * w_scales[c]
// with 16x16x64 integer matrix instructions.  The sums are exact, so any order of K
// gives the same bits.
//
// A workgroup takes one tile of 16 columns and up to 64 rows over the whole of K,
// its waves every so-many-th fragment of the tile, and adds the waves' sums through
// LDS.  The weight is the instruction's first operand: a lane ends with four
// neighbouring columns of one row.
#include <hip/hip_runtime.h>

#include "i8_device.h"

namespace dspk {
namespace {

using namespace i8;

// One 16-byte piece of the tiles per thread.
__global__ __launch_bounds__(256) void i8_pack_kernel(const I8PackArgs A) {
    const int64_t pieces = A.tiles * A.steps * 64;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * 256) {
        const int lane = (int)(i & 63);
        const int64_t frag = i >> 6, tile = frag / A.steps, g = tile / A.tiles_n;
        const int r0 = (int)(frag - tile * A.steps) * kI8K + 16 * (lane >> 4);
        const int col = (int)(tile - g * A.tiles_n) * kI8Cols + (lane & 15);
        const int8_t *src = A.codes + (g * A.n + col) * A.ldc + r0;
        u32x4 v = {0u, 0u, 0u, 0u};
        if (col < A.n)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (r0 + e < A.k) v[e / 4] |= (uint32_t)(uint8_t)src[e] << (8 * (e % 4));
        ((u32x4 *)A.out)[i] = v;
    }
}

// MT 16-row tiles; U fragments of a wave on their way at a time.
template <int MT, int U, bool BF16>
__global__ __launch_bounds__(1024) void i8_gemm_kernel(const I8GemmArgs A) {
    extern __shared__ i32x4 part[];                // [wave][MT][lane]
    const int lane = threadIdx.x & 63, c = lane & 15, j = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int row0 = blockIdx.y * 16 * MT;
    const char *wt = A.tiles + (int64_t)blockIdx.x * A.steps * kI8Frag + 16 * lane;
    const int8_t *xr[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) xr[i] = A.x + (int64_t)min(row0 + 16 * i + c, A.m - 1) * A.ldx;
    i32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = i32x4{0, 0, 0, 0};
    for (int s0 = w; s0 < A.steps; s0 += U * waves) {
        i32x4 f[U], x[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // past the last fragment: that one again, as zeros
            const int s = s0 + u * waves, at = min(s, A.steps - 1);
            f[u] = __builtin_nontemporal_load((const i32x4 *)(wt + (int64_t)at * kI8Frag));
            if (s >= A.steps) f[u] = i32x4{0, 0, 0, 0};
            const int r = at * kI8K + 16 * j, rr = r < A.k ? r : 0;     // past k the weight is zero
#pragma unroll
            for (int i = 0; i < MT; ++i) x[u][i] = *(const i32x4 *)(xr[i] + rr);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[i] = mfma64(f[u], x[u][i], acc[i]);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) part[(w * MT + i) * 64 + lane] = acc[i];
    __syncthreads();
    for (int q = threadIdx.x; q < MT * 64; q += blockDim.x) {
        i32x4 sum = part[q];
        for (int i = 1; i < waves; ++i) sum += part[i * MT * 64 + q];
        const int row = row0 + 16 * (q >> 6) + (q & 15), col = blockIdx.x * kI8Cols + 4 * ((q >> 4) & 3);
        if (row >= A.m) continue;
        const float xs = A.x_scales[row];
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = col + e < A.n ? (float)sum[e] * xs * A.w_scales[col + e] : 0.f;
        store4<BF16>(A.y, row * A.ldy + col, col, A.n, A.vec, v);
    }
}

template <int MT, int U>
hipError_t launch_mt(const I8GemmArgs &a, const I8Plan &p, hipStream_t s) {
    const dim3 grid((unsigned)p.grid_x, (unsigned)p.grid_y), block(64 * p.waves);
    const size_t lds = (size_t)p.waves * MT * 1024;
    if (a.y_bf16)
        hipLaunchKernelGGL((i8_gemm_kernel<MT, U, true>), grid, block, lds, s, a);
    else
        hipLaunchKernelGGL((i8_gemm_kernel<MT, U, false>), grid, block, lds, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_pack(const I8PackArgs &a, hipStream_t s) {
    const int64_t blocks = (a.tiles * a.steps * 64 + 255) / 256;
    hipLaunchKernelGGL(i8_pack_kernel, dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20)), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_i8_gemm(const I8GemmArgs &a, const I8Plan &p, hipStream_t s) {
    switch (p.row_tiles) {
        case 1: return launch_mt<1, 8>(a, p, s);
        case 2: return launch_mt<2, 4>(a, p, s);
        case 4: return launch_mt<4, 4>(a, p, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace dspk
