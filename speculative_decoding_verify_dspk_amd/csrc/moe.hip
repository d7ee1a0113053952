// A mixture-of-experts layer for a few tokens: the router, and the experts in two
// launches.
//
//   route  scores of 16 experts per workgroup (bf16 matrix instructions, K split
//          over its waves); the last workgroup to arrive chooses, a wave per row.
//   up     a workgroup per chosen expert and 16 columns of gate and up, over the
//          tokens that chose it: h = silu(gate) * up in fp32, the largest |h| of each
//          row by atomic maximum (which no order changes).
//   down   a workgroup per chosen expert and 64 columns of down: h's rows to codes
//          in LDS, products, then the last workgroup of a column block adds
//          the slots of each token in their order.
// Which experts are chosen is found by every workgroup for itself from ids: the
// launch has as many as could be, those past the chosen ones end.  Each expert's
// weights are read once for up to 32 of its rows.
#include <hip/hip_runtime.h>

#include "i8_device.h"

namespace dspk {
namespace {

using namespace i8;

typedef __attribute__((ext_vector_type(4))) float f4;

// ---------------------------------------------------------------------- route
constexpr int kRouteWaves = 8;

// Eight bf16 of a row from column r on, those at k and past it zeros.
__device__ __forceinline__ bf16x8 bf16_piece(const uint16_t *row, int r, int k) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (r < k) {
        v = *(const u32x4 *)(row + r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (r + 2 * e >= k) v[e] = 0u;
            else if (r + 2 * e + 1 >= k) v[e] &= 0xffffu;
        }
    }
    return __builtin_bit_cast(bf16x8, v);
}

// Scores ordered as integers: larger score, larger key; NaN below all.  Zeros of
// both signs are one score.
__device__ __forceinline__ uint32_t score_key(float z) {
    if (!(z == z)) return 0u;
    const uint32_t b = __float_as_uint(z + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A wave's choice for one row: NV scores per lane, expert 64 i + lane.
template <int NV>
__device__ __forceinline__ void choose(const RouteArgs &A, int row, int lane) {
    float z[NV];
    uint64_t key[NV];
    bool bad = false;
    float most = -__uint_as_float(0x7f800000u);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = 64 * i + lane;
        z[i] = 0.f;
        key[i] = 0;
        if (e < A.experts) {
            z[i] = __hip_atomic_load(A.part + (int64_t)row * A.experts + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            bad |= !(z[i] == z[i]);
            most = fmaxf(most, z[i]);
            // every expert's key is above 0; of equal scores the lower expert's is larger
            key[i] = (uint64_t)score_key(z[i]) << 32 | (uint32_t)(kMoeMaxExperts - e);
        }
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) most = fmaxf(most, __shfl_xor(most, o));
    bad = __any(bad);
    float sum = 0.f;
    if (!A.normalize) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (64 * i + lane < A.experts) sum += expf(z[i] - most);
#pragma unroll
        for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
    }
    float mine = 0.f;                              // lane j's weight: slot j's
    int id = 0;
    for (int j = 0; j < A.top_k; ++j) {
        uint64_t best = key[0];
        float bz = z[0];
#pragma unroll
        for (int i = 1; i < NV; ++i)
            if (key[i] > best) best = key[i], bz = z[i];
        const uint64_t own = best;
#pragma unroll
        for (int o = 32; o; o >>= 1) {
            const uint64_t other = (uint64_t)__shfl_xor((unsigned long long)best, o);
            best = other > best ? other : best;
        }
        const int from = __ffsll((unsigned long long)__ballot(own == best)) - 1;
        const float p = expf(__shfl(bz, from) - most);
        if (A.normalize) sum += p;
        if (lane == j) mine = p, id = kMoeMaxExperts - (int)(uint32_t)best;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (key[i] == best) key[i] = 0;
    }
    if (lane < A.top_k) {
        A.ids[row * A.top_k + lane] = id;
        A.weights[row * A.top_k + lane] = bad ? __uint_as_float(0x7fc00000u) : mine / sum;
    }
}

template <int MT>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(const RouteArgs A) {
    __shared__ f4 part[kRouteWaves][MT][64];
    const int lane = threadIdx.x & 63, c = lane & 15, j = lane >> 4, w = threadIdx.x >> 6;
    const int e0 = blockIdx.x * 16;
    const uint16_t *rr = A.router + (int64_t)min(e0 + c, A.experts - 1) * A.ldr;
    f4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = f4{0.f, 0.f, 0.f, 0.f};
    for (int r0 = 32 * w; r0 < A.k; r0 += 32 * kRouteWaves) {
        const bf16x8 a = bf16_piece(rr, r0 + 8 * j, A.k);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const bf16x8 b = bf16_piece(A.x + (int64_t)min(16 * i + c, A.m - 1) * A.ldx, r0 + 8 * j, A.k);
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc[i], 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) part[w][i][lane] = acc[i];
    __syncthreads();
    for (int q = threadIdx.x; q < MT * 64; q += blockDim.x) {
        f4 z = part[0][q >> 6][q & 63];
        for (int i = 1; i < kRouteWaves; ++i) z += part[i][q >> 6][q & 63];
        const int row = 16 * (q >> 6) + (q & 15), e = e0 + 4 * ((q >> 4) & 3);
        if (row < A.m)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (e + k < A.experts) {
                    __hip_atomic_store(A.part + (int64_t)row * A.experts + e + k, z[k], __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
                    if (A.scores != nullptr) A.scores[row * A.lds + e + k] = z[k];
                }
    }
    if (!last_to_arrive(A.counter, gridDim.x)) return;
    for (int row = w; row < A.m; row += kRouteWaves) {
        if (A.experts <= 128)
            choose<2>(A, row, lane);
        else if (A.experts <= 256)
            choose<4>(A, row, lane);
        else
            choose<kMoeMaxExperts / 64>(A, row, lane);
    }
}

// -------------------------------------------------------------------- experts
constexpr int kMoeWaves = 4, kMoeThreads = 64 * kMoeWaves;

// What a workgroup knows of the choice: how many experts were chosen, which its own is
// (-1: none), and the slots (token * top_k + j) that chose it.
struct Chosen {
    uint32_t map[kMoeMaxExperts / 32];
    int32_t count;                                 // slots of this expert
    uint16_t slots[kMoeMaxSlots];
};
__device__ __forceinline__ int find(Chosen &S, const MoeArgs &A, int index, int &active) {
    const int slots = A.m * A.top_k, t = threadIdx.x;
    if (t < kMoeMaxExperts / 32) S.map[t] = 0u;
    if (t == 0) S.count = 0;
    __syncthreads();
    for (int i = t; i < slots; i += kMoeThreads) {
        const uint32_t e = (uint32_t)A.ids[i];
        if (e < (uint32_t)A.experts) atomicOr(&S.map[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    int mine = -1;
    active = 0;
    for (int i = 0; 32 * i < A.experts; ++i) {
        uint32_t bits = S.map[i];
        const int n = __popc(bits);
        if (index >= active && index < active + n) {
            for (int skip = index - active; skip; --skip) bits &= bits - 1;
            mine = 32 * i + __ffs(bits) - 1;
        }
        active += n;
    }
    if (mine < 0) return -1;
    // in any order: a row's result does not depend on its place
    for (int i = t; i < slots; i += kMoeThreads)
        if (A.ids[i] == mine) S.slots[atomicAdd(&S.count, 1)] = (uint16_t)i;
    __syncthreads();
    return mine;
}

// Rows [base, base + 16 MT) of the expert's list.
template <int MT>
__device__ __forceinline__ void up_rows(const MoeArgs &A, const Chosen &S, int base, const char *gt, const char *ut,
                                        const float *gs, const float *us, int steps, i32x4 (*part)[4][64]) {
    constexpr int U = 4;
    const int lane = threadIdx.x & 63, c = lane & 15, j = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int8_t *xr[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
        xr[i] = A.x + (int64_t)(S.slots[min(base + 16 * i + c, S.count - 1)] / (uint32_t)A.top_k) * A.ldx;
    i32x4 g[MT], u[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) g[i] = u[i] = i32x4{0, 0, 0, 0};
    for (int s0 = w; s0 < steps; s0 += U * kMoeWaves) {
        i32x4 fg[U], fu[U], x[U][MT];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int s = s0 + q * kMoeWaves, at = min(s, steps - 1);
            fg[q] = *(const i32x4 *)(gt + (int64_t)at * kI8Frag);
            fu[q] = *(const i32x4 *)(ut + (int64_t)at * kI8Frag);
            if (s >= steps) fg[q] = fu[q] = i32x4{0, 0, 0, 0};
            const int r = at * kI8K + 16 * j, rr = r < A.hidden ? r : 0;
#pragma unroll
            for (int i = 0; i < MT; ++i) x[q][i] = *(const i32x4 *)(xr[i] + rr);
        }
#pragma unroll
        for (int q = 0; q < U; ++q)
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                g[i] = mfma64(fg[q], x[q][i], g[i]);
                u[i] = mfma64(fu[q], x[q][i], u[i]);
            }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) part[w][2 * i][lane] = g[i], part[w][2 * i + 1][lane] = u[i];
    __syncthreads();
    if (w < MT && base + 16 * w < S.count) {       // wave w: row tile w
        i32x4 a = part[0][2 * w][lane], b = part[0][2 * w + 1][lane];
#pragma unroll
        for (int i = 1; i < kMoeWaves; ++i) a += part[i][2 * w][lane], b += part[i][2 * w + 1][lane];
        const int at = base + 16 * w + c, slot = S.slots[min(at, S.count - 1)];
        const float xs = A.x_scales[slot / (uint32_t)A.top_k];
        const int col = blockIdx.x * kI8Cols + 4 * j;
        f4 h;
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            h[e] = col + e < A.inter ? silu((float)a[e] * xs * gs[col + e]) * ((float)b[e] * xs * us[col + e]) : 0.f;
            top = max(top, magnitude(h[e]));
        }
        if (at < S.count) *(f4 *)(A.h + (int64_t)slot * A.ldh + col) = h;
        top = max(top, (uint32_t)__shfl_xor((int)top, 16));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        if (at < S.count && j == 0) atomicMax(A.top + slot, top);
    }
    __syncthreads();
}

__global__ __launch_bounds__(kMoeThreads) void moe_up_kernel(const MoeArgs A) {
    __shared__ Chosen S;
    __shared__ i32x4 part[kMoeWaves][4][64];
    int active;
    const int e = find(S, A, blockIdx.y, active);
    if (e < 0) return;
    const int steps = (int)i8_steps(A.hidden), tiles = gridDim.x;
    const int64_t tile = ((int64_t)e * tiles + blockIdx.x) * steps * kI8Frag + 16 * (threadIdx.x & 63);
    const float *gs = A.gate_scales + (int64_t)e * A.inter, *us = A.up_scales + (int64_t)e * A.inter;
    for (int base = 0; base < S.count; base += 32) {
        if (S.count - base <= 16)
            up_rows<1>(A, S, base, A.gate + tile, A.up + tile, gs, us, steps, part);
        else
            up_rows<2>(A, S, base, A.gate + tile, A.up + tile, gs, us, steps, part);
    }
}

constexpr int kMoeChunk = 1024;     // K of h's codes in LDS at a time

template <int MT>
__device__ __forceinline__ void down_rows(const MoeArgs &A, const Chosen &S, int base, const char *dt, const float *ds,
                                          int tile, int tiles, int steps, i32x4 *codes, const Step8 *st) {
    constexpr int U = 4;
    const int lane = threadIdx.x & 63, c = lane & 15, j = lane >> 4;
    const int rows = min(S.count - base, 16 * MT);
    i32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = i32x4{0, 0, 0, 0};
    for (int k0 = 0; k0 < A.inter; k0 += kMoeChunk) {
        const int pieces = min(kMoeChunk, (int)A.ldh - k0) / 16;       // 16-column pieces of a row, ldh is whole ones
        const int n = min(kMoeChunk / kI8K, steps - k0 / kI8K);
        __syncthreads();                           // the chunk before has been read
        for (int p = threadIdx.x; p < rows * pieces; p += kMoeThreads) {
            const int r = p / pieces, q = p - r * pieces;
            const f4 *src = (const f4 *)(A.h + (int64_t)S.slots[base + r] * A.ldh + k0 + 16 * q);
            const Step8 s = st[r];
            i32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f4 h = src[e];
                v[e] = (int32_t)codes8(h[0], h[1], h[2], h[3], s);
            }
            codes[((q >> 2) * MT + (r >> 4)) * 64 + (q & 3) * 16 + (r & 15)] = v;
        }
        __syncthreads();
        if (tile < tiles)
            for (int s0 = 0; s0 < n; s0 += U) {
                i32x4 f[U];
#pragma unroll
                for (int q = 0; q < U; ++q)
                    f[q] = *(const i32x4 *)(dt + (int64_t)(k0 / kI8K + min(s0 + q, n - 1)) * kI8Frag);
#pragma unroll
                for (int q = 0; q < U; ++q)
                    if (s0 + q < n)
#pragma unroll
                        for (int i = 0; i < MT; ++i)
                            acc[i] = mfma64(f[q], codes[((s0 + q) * MT + i) * 64 + lane], acc[i]);
            }
    }
    if (tile >= tiles) return;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int r = 16 * i + c, col = tile * kI8Cols + 4 * j;
        if (r >= rows) continue;
        const float hs = st[r].scale;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = col + e < A.hidden ? (float)acc[i][e] * hs * ds[col + e] : 0.f;
        float *p = A.part + (int64_t)S.slots[base + r] * A.ldp + col;
        share(p, v[0], v[1]);
        share(p + 2, v[2], v[3]);
    }
}

template <bool BF16>
__global__ __launch_bounds__(kMoeThreads) void moe_down_kernel(const MoeArgs A) {
    __shared__ Chosen S;
    __shared__ i32x4 codes[2 * kMoeChunk / kI8K * 64];
    __shared__ Step8 st[32];
    int active;
    const int e = find(S, A, blockIdx.y, active);
    // with no expert chosen at all the first row of workgroups still writes y
    if (e < 0 && !(active == 0 && blockIdx.y == 0)) return;
    const int steps = (int)i8_steps(A.inter), tiles = (int)i8_tiles(A.hidden);
    if (e >= 0) {
        const int tile = blockIdx.x * (kMoeCols / kI8Cols) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const char *dt = A.down + ((int64_t)e * tiles + min(tile, tiles - 1)) * steps * kI8Frag + 16 * (threadIdx.x & 63);
        const float *ds = A.down_scales + (int64_t)e * A.hidden;
        for (int base = 0; base < S.count; base += 32) {
            __syncthreads();
            if (threadIdx.x < 32) st[threadIdx.x] = step8(A.top[S.slots[min(base + (int)threadIdx.x, S.count - 1)]]);
            __syncthreads();
            if (S.count - base <= 16)
                down_rows<1>(A, S, base, dt, ds, tile, tiles, steps, codes, st);
            else
                down_rows<2>(A, S, base, dt, ds, tile, tiles, steps, codes, st);
        }
    }
    if (!last_to_arrive(A.ctr + blockIdx.x, max(active, 1))) return;
    // this column block's products are all there: each token's slots in their order
    for (int i = threadIdx.x; i < A.m * (kMoeCols / 2); i += kMoeThreads) {
        const int row = i / (kMoeCols / 2), col = blockIdx.x * kMoeCols + 2 * (i % (kMoeCols / 2));
        if (col >= A.hidden) continue;
        float a = 0.f, b = 0.f;
        for (int q = 0; q < A.top_k; ++q) {
            const int slot = row * A.top_k + q, id = A.ids[slot];
            if (id == -1) continue;
            float2 p = make_float2(__uint_as_float(0x7fc00000u), __uint_as_float(0x7fc00000u));
            if ((uint32_t)id < (uint32_t)A.experts) p = shared2(A.part + (int64_t)slot * A.ldp + col);
            const float wt = A.weights[slot];
            a += wt * p.x;
            b += wt * p.y;
        }
        const int64_t at = row * A.ldy + col;
        if constexpr (BF16) {
            ((uint16_t *)A.y)[at] = to_bf16(a);
            if (col + 1 < A.hidden) ((uint16_t *)A.y)[at + 1] = to_bf16(b);
        } else {
            ((float *)A.y)[at] = a;
            if (col + 1 < A.hidden) ((float *)A.y)[at + 1] = b;
        }
    }
    // the last column block: every workgroup has read the largest magnitudes
    if (!last_to_arrive(A.done, gridDim.x)) return;
    for (int i = threadIdx.x; i < A.m * A.top_k; i += kMoeThreads) A.top[i] = 0u;
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs &a, hipStream_t s) {
    const dim3 grid((a.experts + 15) / 16), block(64 * kRouteWaves);
    if (a.m <= 16)
        hipLaunchKernelGGL((route_kernel<1>), grid, block, 0, s, a);
    else if (a.m <= 32)
        hipLaunchKernelGGL((route_kernel<2>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((route_kernel<4>), grid, block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_moe_mlp(const MoeArgs &a, hipStream_t s) {
    const int slots = a.m * a.top_k, most = slots < a.experts ? slots : a.experts;
    hipLaunchKernelGGL(moe_up_kernel, dim3((a.inter + kI8Cols - 1) / kI8Cols, most), dim3(kMoeThreads), 0, s, a);
    const dim3 grid((a.hidden + kMoeCols - 1) / kMoeCols, most);
    if (a.y_bf16)
        hipLaunchKernelGGL((moe_down_kernel<true>), grid, dim3(kMoeThreads), 0, s, a);
    else
        hipLaunchKernelGGL((moe_down_kernel<false>), grid, dim3(kMoeThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace dspk
