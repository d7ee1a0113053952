// Row kernels of the 8-bit integer side: a workgroup takes a row, each lane pieces
// of eight neighbouring columns that stay in registers from the one load to the
// one store.
//   norm   s = x + residual, residual_out = s, y = (s * w) * (1 / sqrt(mean(s^2) + eps))
//   silu   y = gate / (1 + exp(-gate)) * up
//   plain  y = x
// with y as bf16 rows, as codes with a scale, or both.  For a norm the scale's
// largest |y| is the largest |s * w| times that factor (a rounded product with
// a positive factor keeps order), so sum of squares and largest magnitude are found
// in one pass over the lanes.
#include <hip/hip_runtime.h>

#include "i8_device.h"

namespace dspk {
namespace {

using namespace i8;

// Eight neighbouring elements, those at `left` and past it zeros.
template <bool F32>
__device__ __forceinline__ void load8(const void *p, int64_t at, int left, float (&v)[8]) {
    if (left >= 8) {
        if constexpr (F32) {
            const f32x4 *q = (const f32x4 *)((const float *)p + at);
            const f32x4 a = q[0], b = q[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
        } else {
            const u32x4 a = *(const u32x4 *)((const uint16_t *)p + at);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[2 * e] = bf16_lo(a[e]), v[2 * e + 1] = bf16_hi(a[e]);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = 0.f;
        if (e < left)
            v[e] = F32 ? ((const float *)p)[at + e] : __uint_as_float((uint32_t)((const uint16_t *)p)[at + e] << 16);
    }
}
template <bool F32>
__device__ __forceinline__ void store8(void *p, int64_t at, int left, const float (&v)[8]) {
    if (left >= 8) {
        if constexpr (F32) {
            f32x4 *q = (f32x4 *)((float *)p + at);
            q[0] = f32x4{v[0], v[1], v[2], v[3]};
            q[1] = f32x4{v[4], v[5], v[6], v[7]};
        } else {
            *(u32x4 *)((uint16_t *)p + at) = u32x4{to_bf16_pair(v[0], v[1]), to_bf16_pair(v[2], v[3]),
                                                   to_bf16_pair(v[4], v[5]), to_bf16_pair(v[6], v[7])};
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < left) {
            if constexpr (F32)
                ((float *)p)[at + e] = v[e];
            else
                ((uint16_t *)p)[at + e] = to_bf16(v[e]);
        }
}

// P pieces per lane.
template <int OP, bool XF, bool RF, int P>
__global__ __launch_bounds__(kRowMostThreads) void rows_kernel(const RowArgs A) {
    __shared__ float sums[2][kRowMostThreads / 64];
    __shared__ uint32_t tops[2][kRowMostThreads / 64];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, waves = blockDim.x >> 6;
    float w[P][8];
    if constexpr (OP == kRowNorm) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int col = kRowPiece * (p * (int)blockDim.x + t);
            if (A.w != nullptr)
                load8<true>(A.w, col, A.n - col, w[p]);
            else
                for (int e = 0; e < 8; ++e) w[p][e] = 1.f;
        }
    }
    int turn = 0;
    for (int row = blockIdx.x; row < A.m; row += gridDim.x, turn ^= 1) {
        float v[P][8];
        float ss = 0.f;
        uint32_t top = 0;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int col = kRowPiece * (p * (int)blockDim.x + t), left = A.n - col;
            float a[8] = {}, b[8] = {};
            if (A.x != nullptr) load8<XF>(A.x, row * A.ldx + col, left, a);
            if constexpr (OP != kRowPlain)
                if (A.r != nullptr) load8<RF>(A.r, row * A.ldr + col, left, b);
            if constexpr (OP == kRowNorm) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    a[e] += b[e];
                    ss += a[e] * a[e];
                    v[p][e] = a[e] * w[p][e];
                }
                if (A.r_out != nullptr) store8<RF>(A.r_out, row * A.ldro + col, left, a);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[p][e] = OP == kRowSilu ? silu(a[e]) * b[e] : a[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, magnitude(v[p][e]));
        }
        float inv = 1.f;
        if (OP == kRowNorm || A.codes != nullptr) {
            if constexpr (OP == kRowNorm) ss = wave_sum(ss);
            top = wave_max(top);
            if (waves > 1) {                       // two sets in turn: the next row's need no second barrier
                if (lane == 0) sums[turn][wave] = ss, tops[turn][wave] = top;
                __syncthreads();
                ss = 0.f, top = 0;
                for (int i = 0; i < waves; ++i) ss += sums[turn][i], top = max(top, tops[turn][i]);
            }
            if constexpr (OP == kRowNorm) {
                inv = 1.f / sqrtf(ss / (float)A.n + A.eps);
                top = magnitude(__uint_as_float(top) * inv);
            }
        }
        const Step8 st = step8(top);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int col = kRowPiece * (p * (int)blockDim.x + t), left = A.n - col;
            if (left <= 0) break;
            if constexpr (OP == kRowNorm)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[p][e] *= inv;
            if (A.rows != nullptr) store8<false>(A.rows, row * A.ld + col, left, v[p]);
            if (A.codes != nullptr) {
                const u32x2 c = {codes8(v[p][0], v[p][1], v[p][2], v[p][3], st),
                                 codes8(v[p][4], v[p][5], v[p][6], v[p][7], st)};
                int8_t *q = A.codes + row * A.ldc + col;
                if (left >= 8)
                    *(u32x2 *)q = c;
                else
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < left) q[e] = (int8_t)(c[e / 4] >> (8 * (e % 4)));
            }
        }
        if (A.codes != nullptr && t == 0) A.scales[row] = st.scale;
    }
}

template <int OP, bool XF, bool RF>
hipError_t launch_p(const RowArgs &a, int cus, hipStream_t s) {
    const int pieces = (a.n + kRowPiece - 1) / kRowPiece;
    const int p = pieces <= 1024 ? 1 : pieces <= 2048 ? 2 : 4;
    const int threads = ((pieces + p - 1) / p + 63) / 64 * 64;
    const int64_t most = (int64_t)cus * (2048 / threads);
    const dim3 grid((unsigned)(a.m < most ? a.m : most)), block(threads);
    if (p == 1)
        hipLaunchKernelGGL((rows_kernel<OP, XF, RF, 1>), grid, block, 0, s, a);
    else if (p == 2)
        hipLaunchKernelGGL((rows_kernel<OP, XF, RF, 2>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((rows_kernel<OP, XF, RF, 4>), grid, block, 0, s, a);
    return hipGetLastError();
}

// 16 codes of a row at a time.
template <bool F32>
__global__ __launch_bounds__(256) void i8_read_kernel(const I8ReadArgs A) {
    const int per = (A.n + 15) / 16;
    const int64_t pieces = (int64_t)A.m * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per;
        const int col = (int)(i - row * per) * 16, left = A.n - col;
        const u32x4 c = *(const u32x4 *)(A.codes + row * A.ldc + col);
        const float s = A.scales[row];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (left <= 8 * h) break;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = s * (float)(int8_t)(c[2 * h + e / 4] >> (8 * (e % 4)));
            store8<F32>(A.y, row * A.ldy + col + 8 * h, left - 8 * h, v);
        }
    }
}

}  // namespace

hipError_t launch_rows(RowOp op, const RowArgs &a, int cus, hipStream_t s) {
    if (op == kRowPlain) return a.x_f32 ? launch_p<kRowPlain, true, true>(a, cus, s) : launch_p<kRowPlain, false, false>(a, cus, s);
    if (op == kRowSilu) return a.x_f32 ? launch_p<kRowSilu, true, true>(a, cus, s) : launch_p<kRowSilu, false, false>(a, cus, s);
    if (a.x_f32) return a.r_f32 ? launch_p<kRowNorm, true, true>(a, cus, s) : launch_p<kRowNorm, true, false>(a, cus, s);
    return a.r_f32 ? launch_p<kRowNorm, false, true>(a, cus, s) : launch_p<kRowNorm, false, false>(a, cus, s);
}

hipError_t launch_i8_read(const I8ReadArgs &a, hipStream_t s) {
    const int64_t pieces = (int64_t)a.m * ((a.n + 15) / 16), blocks = (pieces + 255) / 256;
    const dim3 grid((unsigned)(blocks < (1 << 16) ? blocks : 1 << 16));
    if (a.y_f32)
        hipLaunchKernelGGL((i8_read_kernel<true>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((i8_read_kernel<false>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace dspk
