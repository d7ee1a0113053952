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
//
// Bound by memory for many rows, by the chain of load, reduction and store (and the
// launch) for few.  Measured: norm of 8190 bf16 rows of 5120 with the residual, 8-bit
// out 66 us (293 MB, 4.4 TB/s; a large copy reaches 5.1), one row of 2560 2.6 us;
// activation of 1500 rows of 9728 21 us (73 MB); 8190 rows of 5120 from bf16 to codes 31 us
// (4.0 TB/s), from fp32 41 (5.2), one of 4096 2.0; from codes to bf16 22 us (126 MB).
// Without the next row on its way the norm takes 88 us.
// Rows over 16384 values take four pieces per lane, for which a lane has no registers where
// an input is fp32: the norm then holds 74 to 266 of them in scratch, the activation 107.
// 2000 rows of 32768: norm of bf16 rows 96 us (4.7 TB/s), of fp32 rows with a bf16 residual
// 172 (3.4); activation of bf16 rows 84 (3.9), of fp32 rows 199 (3.0).
#include <hip/hip_runtime.h>

#include "i8_device.h"

namespace dspk {
namespace {

using namespace i8;

// Eight neighbouring elements as they lie in memory, those at `left` and past it zeros.
template <bool F32>
struct Piece {
    u32x4 v[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *p, int64_t at, int left) {
        const char *q = (const char *)p + at * (F32 ? 4 : 2);
        if (left >= 8) {
            v[0] = *(const u32x4 *)q;
            if constexpr (F32) v[1] = *(const u32x4 *)(q + 16);
            return;
        }
        v[0] = u32x4{0u, 0u, 0u, 0u};
        if constexpr (F32) v[1] = v[0];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left) {
                if constexpr (F32)
                    v[e / 4][e % 4] = ((const uint32_t *)q)[e];
                else
                    v[0][e / 2] |= (uint32_t)((const uint16_t *)q)[e] << (16 * (e % 2));
            }
    }
    __device__ __forceinline__ float get(int e) const {
        if constexpr (F32) return __uint_as_float(v[e / 4][e % 4]);
        else return e % 2 ? bf16_hi(v[0][e / 2]) : bf16_lo(v[0][e / 2]);
    }
};
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

// P pieces per lane.  A row's pieces are on their way while the row before is worked on.
template <int OP, bool XF, bool RF, int P>
__global__ __launch_bounds__(kRowMostThreads) void rows_kernel(const RowArgs A) {
    __shared__ float sums[2][kRowMostThreads / 64];
    __shared__ uint32_t tops[2][kRowMostThreads / 64];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, waves = blockDim.x >> 6;
    Piece<true> w[P];
    Piece<XF> x[P];
    Piece<RF> r[P];
    auto fetch = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int col = kRowPiece * (p * (int)blockDim.x + t), left = A.n - col;
            if (A.x != nullptr) x[p].load(A.x, row * A.ldx + col, left);
            if constexpr (OP != kRowPlain)
                if (A.r != nullptr) r[p].load(A.r, row * A.ldr + col, left);
        }
    };
    uint32_t row = blockIdx.x;
    fetch(row);
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int col = kRowPiece * (p * (int)blockDim.x + t);
        if constexpr (OP == kRowNorm)
            if (A.w != nullptr) w[p].load(A.w, col, A.n - col);
    }
    for (int turn = 0;; turn ^= 1) {               // the grid has no more workgroups than rows
        float v[P][8];
        float ss = 0.f;
        uint32_t top = 0;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int col = kRowPiece * (p * (int)blockDim.x + t), left = A.n - col;
            float s[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float a = A.x != nullptr ? x[p].get(e) : 0.f;
                if constexpr (OP == kRowNorm) {
                    s[e] = a + (A.r != nullptr ? r[p].get(e) : 0.f);
                    ss += s[e] * s[e];
                    v[p][e] = A.w != nullptr ? s[e] * w[p].get(e) : s[e];
                } else {
                    v[p][e] = OP == kRowSilu ? silu(a) * r[p].get(e) : a;
                }
                top = max(top, magnitude(v[p][e]));
            }
            if constexpr (OP == kRowNorm)
                if (A.r_out != nullptr) store8<RF>(A.r_out, row * A.ldro + col, left, s);
        }
        const uint32_t next = row + gridDim.x;     // below 2^32: rows and workgroups are below 2^31
        const bool more = next < (uint32_t)A.m;
        if (more) fetch(next);
        float inv = 1.f;
        if (OP == kRowNorm || A.codes != nullptr) {
            float all = OP == kRowNorm ? wave_sum(ss) : 0.f;
            top = wave_max(top);
            if (waves > 1) {                       // two sets in turn: the next row's need no second barrier
                if (lane == 0) sums[turn][wave] = all, tops[turn][wave] = top;
                __syncthreads();
                all = 0.f, top = 0;
                for (int i = 0; i < waves; ++i) all += sums[turn][i], top = max(top, tops[turn][i]);
            }
            if constexpr (OP == kRowNorm) {
                float mean = all / (float)A.n;
                // Squares of 1e18 pass fp32's largest number from 341 of them on, a lane's 32 do
                // not: the lanes' sums are added up again, 2^-8 times as large.
                // (Said to be rare where nothing spills: 6 rows of 2560 2.77 -> 2.74 us, but two of
                // 32768 15.9 -> 17.0.)
                const bool far = __float_as_uint(all) == 0x7f800000u;
                if (P == 4 ? far : __builtin_expect(far, 0)) {
                    all = wave_sum(ss * 0x1p-8f);
                    if (waves > 1) {
                        __syncthreads();
                        if (lane == 0) sums[turn][wave] = all;
                        __syncthreads();
                        all = 0.f;
                        for (int i = 0; i < waves; ++i) all += sums[turn][i];
                    }
                    mean = all / (float)A.n * 0x1p8f;
                }
                inv = 1.f / sqrtf(mean + A.eps);
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
        if (!more) break;
        row = next;
    }
}

template <int OP, bool XF, bool RF>
hipError_t launch_p(const RowArgs &a, int cus, hipStream_t s) {
    const int pieces = (a.n + kRowPiece - 1) / kRowPiece;
    const int p = pieces <= 1024 ? 1 : pieces <= 2048 ? 2 : 4;
    const int threads = ((pieces + p - 1) / p + 63) / 64 * 64;
    // twice the threads a CU holds (8190 rows of 5120: 66 us; as many as it holds 77)
    const int64_t most = (int64_t)cus * 4096 / threads;
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
