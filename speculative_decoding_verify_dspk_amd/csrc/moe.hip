// A mixture-of-experts layer for a few tokens: the router, and the experts in two
// launches.
//
//   route  scores of 16 experts per workgroup (bf16 matrix instructions, K split
//          over its waves); the last workgroup to arrive chooses, a wave per row.
//   up     a workgroup per chosen expert and 32 columns of gate and up, over the
//          tokens that chose it: h = silu(gate) * up in fp32.
//   down   a workgroup per 16 columns of y: its waves share out the chosen experts and
//          their K, add whole-number sums in LDS (exact in any order), and then each
//          token's slots in their order.
// Between them h's rows become codes: few and short ones in every down workgroup for
// itself, while its weights are on their way; else in the last of an expert's up
// workgroups to arrive (some 3 us of stores, arrivals and loads that pass between dies).
// An expert's gate and up are read once for up to 32 of its rows, its down once for up to
// 16 of those in a group of slots; more rows read them again.
//
// Bound by the chosen experts' way from memory where there are many, by chains of
// dependent accesses where there are few.  Measured (us): 1 / 6 rows of 8 of 128 experts
// 2048 -> 768 (38 / some 190 MB): route 7.2 / 8.2, up 7.7 / 27.0, down 6.9 / 16.7; 32 rows of 2 of
// 8, 4096 -> 14336 (1409 MB): route 6.8, up 167 (5.6 TB/s), down 76 (6.2; a large copy
// moves 5.1, half of it stores).
#include <hip/hip_runtime.h>

#include "i8_device.h"

namespace dspk {
namespace {

using namespace i8;

typedef __attribute__((ext_vector_type(4))) float f4;

// ---------------------------------------------------------------------- route
constexpr int kRouteWaves = 16;

// Eight bf16 of a row from column r on, those at k and past it zeros.  Columns are numbered
// in 32 unsigned bits: k is below 2^31, and the router's waves stop within a few thousand
// columns of it.
__device__ __forceinline__ bf16x8 bf16_piece(const uint16_t *row, uint32_t r, uint32_t k) {
    u32x4 v = *(const u32x4 *)(row + (r < k ? r : 0));     // no branch: several are on their way
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = r + 2 * e + 1 < k ? v[e] : r + 2 * e < k ? v[e] & 0xffffu : 0u;
    return __builtin_bit_cast(bf16x8, v);
}

// Scores ordered as integers above 0: larger score, larger key; NaN below all.  Zeros
// of both signs are one score.
__device__ __forceinline__ uint32_t score_key(float z) {
    if (!(z == z)) return 1u;
    const uint32_t b = __float_as_uint(z + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_score(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);    // 1 gives a NaN
}

// A wave's choice for one row: NV scores per lane, score(e) of expert e = 64 i + lane.
template <int NV, class Score>
__device__ __forceinline__ void choose_of(const RouteArgs &A, int row, int lane, const Score &score) {
    float z[NV];
    uint32_t key[NV];                              // 0: no expert, or taken; the others are larger
    bool bad = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = 64 * i + lane;
        z[i] = -__uint_as_float(0x7f800000u);
        if (e < A.experts) z[i] = score(e);
        bad |= !(z[i] == z[i]);
        key[i] = e < A.experts ? score_key(z[i]) : 0u;
    }
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) most = max(most, key[i]);
    most = wave_max(most);
    const float zmost = key_score(most);           // NaN: all are
    bad = __any(bad);
    float sum = 0.f;
    if (!A.normalize) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (64 * i + lane < A.experts) sum += expf(z[i] - zmost);
        sum = wave_sum(sum);
    }
    float mine = 0.f;                              // lane j's: slot j's
    int id = 0;
    for (int j = 0; j < A.top_k; ++j) {
        uint32_t best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < NV; ++i)
            if (key[i] > best) best = key[i], at = i;
        const uint32_t top = wave_max(best);
        // of equal scores the lowest expert: the lowest i, then the lowest lane
        uint64_t same = __ballot(best == top);
        int e = 64 * __builtin_amdgcn_readlane(at, __ffsll((unsigned long long)same) - 1) + __ffsll((unsigned long long)same) - 1;
        for (same &= same - 1; same; same &= same - 1) {
            const int from = __ffsll((unsigned long long)same) - 1;
            e = min(e, 64 * __builtin_amdgcn_readlane(at, from) + from);
        }
        const float p = expf(key_score(top) - zmost);
        if (A.normalize) sum += p;
        if (lane == j) mine = p, id = e;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (64 * i + lane == e) key[i] = 0u;
    }
    if (lane < A.top_k) {
        A.ids[row * A.top_k + lane] = id;
        A.weights[row * A.top_k + lane] = bad ? __uint_as_float(0x7fc00000u) : mine / sum;
    }
}

template <class Score>
__device__ __forceinline__ void choose(const RouteArgs &A, int row, int lane, const Score &score) {
    if (A.experts <= 128)
        choose_of<2>(A, row, lane, score);
    else if (A.experts <= 256)
        choose_of<4>(A, row, lane, score);
    else
        choose_of<kMoeMaxExperts / 64>(A, row, lane, score);
}

// Small routers: a workgroup per row takes all experts, 16 of them to a wave and the
// rest of the waves to parts of K, and nothing has to pass between workgroups (which
// takes some 4 us).
__global__ __launch_bounds__(64 * kRouteWaves) void route_row_kernel(const RouteArgs A) {
    constexpr int U = 8;
    __shared__ float part[kRouteWaves * 16 > kMoeMaxExperts ? kRouteWaves * 16 : kMoeMaxExperts];
    const int lane = threadIdx.x & 63, c = lane & 15, j = lane >> 4, row = blockIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = (A.experts + 15) / 16, ks = tiles >= kRouteWaves ? 1 : kRouteWaves / tiles;
    const uint16_t *const xr = A.x + row * A.ldx;
    for (int item = w; item < tiles * ks; item += kRouteWaves) {
        const int k0 = item / tiles, tile = item - k0 * tiles;
        const uint16_t *const rr = A.router + (int64_t)min(16 * tile + c, A.experts - 1) * A.ldr;
        f4 acc = {0.f, 0.f, 0.f, 0.f};
        for (uint32_t r0 = 32 * k0; r0 < (uint32_t)A.k; r0 += 32 * ks * U) {
            bf16x8 a[U], b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                a[u] = bf16_piece(rr, r0 + 32 * ks * u + 8 * j, A.k);
                b[u] = bf16_piece(xr, r0 + 32 * ks * u + 8 * j, A.k);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[u], b[u], acc, 0, 0, 0);
        }
        if (c == 0)                                // every column of the product is this row
#pragma unroll
            for (int q = 0; q < 4; ++q) part[k0 * 16 * tiles + 16 * tile + 4 * j + q] = acc[q];
    }
    __syncthreads();
    if (w != 0) return;
    choose(A, row, lane, [&](int e) {
        float z = part[e];
        for (int i = 1; i < ks; ++i) z += part[i * 16 * tiles + e];
        if (A.scores != nullptr) A.scores[row * A.lds + e] = z;
        return z;
    });
}

// Scores of 16 experts per workgroup, K by turns over its waves; the last to arrive
// chooses.
template <int MT>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(const RouteArgs A) {
    constexpr int U = MT == 1 ? 4 : 2;             // pieces on their way at a time
    __shared__ f4 part[kRouteWaves][MT][64];
    const int lane = threadIdx.x & 63, c = lane & 15, j = lane >> 4, w = threadIdx.x >> 6;
    const int e0 = blockIdx.x * 16, step = 32 * kRouteWaves;
    const uint16_t *rr = A.router + (int64_t)min(e0 + c, A.experts - 1) * A.ldr;
    const uint16_t *xr[MT];
    f4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        acc[i] = f4{0.f, 0.f, 0.f, 0.f};
        xr[i] = A.x + (int64_t)min(16 * i + c, A.m - 1) * A.ldx;
    }
    for (uint32_t r0 = 32 * w; r0 < (uint32_t)A.k; r0 += step * U) {
        bf16x8 a[U], b[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t r = r0 + step * u + 8 * j;
            a[u] = bf16_piece(rr, r, A.k);
#pragma unroll
            for (int i = 0; i < MT; ++i) b[u][i] = bf16_piece(xr[i], r, A.k);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < MT; ++i)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[u], b[u][i], acc[i], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) part[w][i][lane] = acc[i];
    __syncthreads();
    for (int q = threadIdx.x; q < MT * 256; q += blockDim.x) {
        const int i = q >> 8, l = (q >> 2) & 63;
        float z = part[0][i][l][q & 3];
        for (int o = 1; o < kRouteWaves; ++o) z += part[o][i][l][q & 3];
        const int row = 16 * i + (l & 15), e = e0 + 4 * (l >> 4) + (q & 3);
        if (row < A.m && e < A.experts)
            __hip_atomic_store(A.part + (int64_t)row * A.experts + e, z, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (!last_to_arrive(A.counter, gridDim.x)) return;
    for (int row = w; row < A.m; row += kRouteWaves)
        choose(A, row, lane, [&](int e) {
            const float z =
                __hip_atomic_load(A.part + (int64_t)row * A.experts + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (A.scores != nullptr) A.scores[row * A.lds + e] = z;
            return z;
        });
}

// -------------------------------------------------------------------- experts

// The slots (token * top_k + j) of [first, last) that chose expert e, listed in `slots`
// by every wave for itself (they write the same), and their number.
__device__ __forceinline__ int slots_of(const int32_t *ids, int e, int first, int last, uint16_t *slots) {
    const int lane = threadIdx.x & 63;
    int count = 0;
    for (int i0 = first; i0 < last; i0 += 64) {
        const int i = i0 + lane;
        const bool hit = i < last && ids[i] == e;
        const uint64_t all = __ballot(hit);
        if (hit) slots[count + __popcll(all & ((1ull << lane) - 1))] = (uint16_t)i;
        count += __popcll(all);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");     // lanes read what others of the wave wrote
    return count;
}

// A wave's fragments s0, s0 + step, .. below `end` of T streams of weight tiles against
// MT 16-row tiles of codes, through a ring of D register sets.
template <int T, int MT, int D>
__device__ __forceinline__ void stream(const char *const (&wt)[T], const int8_t *const (&xr)[MT], int k, int s0, int step,
                                       int end, i32x4 (&acc)[T][MT]) {
    const int lane = threadIdx.x & 63, j = lane >> 4;
    struct Set {
        i32x4 f[T], x[MT];
    };
    auto load = [&](int s, Set &o) __attribute__((always_inline)) {
        const int at = min(s, end - 1), r = at * kI8K + 16 * j, in = r < k ? r : 0;      // past k: meets zeros
#pragma unroll
        for (int t = 0; t < T; ++t)
            o.f[t] = __builtin_nontemporal_load((const i32x4 *)(wt[t] + (int64_t)at * kI8Frag + 16 * lane));
#pragma unroll
        for (int i = 0; i < MT; ++i) o.x[i] = *(const i32x4 *)(xr[i] + in);
    };
    auto multiply = [&](int s, const Set &o) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const i32x4 f = s < end ? o.f[t] : i32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[t][i] = mfma64(f, o.x[i], acc[t][i]);
        }
    };
    if (s0 >= end) return;
    Set ring[D];
#pragma unroll
    for (int u = 0; u < D; ++u) load(s0 + u * step, ring[u]);
    __builtin_amdgcn_sched_barrier(0);
    for (; s0 + D * step < end; s0 += D * step) {
#pragma unroll
        for (int u = 0; u < D; ++u) {
            multiply(s0 + u * step, ring[u]);
            load(s0 + (D + u) * step, ring[u]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int u = 0; u < D; ++u) multiply(s0 + u * step, ring[u]);
}

// Rows [base, base + 16 MT) of the expert's list into h, CT tiles of 16 columns from
// `tile0` on.  INSIDE: they become codes inside the down workgroups.
template <int CT, int MT, int W, bool INSIDE>
__device__ __forceinline__ void up_rows(const MoeArgs &A, const uint16_t *slots, int count, int base, int e, int tile0,
                                        int tiles, i32x4 (*part)[2 * CT * 2][64], float *scales) {
    int lane = threadIdx.x & 63, c = lane & 15, j = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), steps = (int)i8_steps(A.hidden);
    const int8_t *xr[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
        xr[i] = A.x + (int64_t)(slots[min(base + 16 * i + c, count - 1)] / (uint32_t)A.top_k) * A.ldx;
    const char *wt[2 * CT];
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        const int64_t at = ((int64_t)e * tiles + min(tile0 + t, tiles - 1)) * steps * kI8Frag;
        wt[2 * t] = A.gate + at;
        wt[2 * t + 1] = A.up + at;
    }
    i32x4 acc[2 * CT][MT];
#pragma unroll
    for (int t = 0; t < 2 * CT; ++t)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[t][i] = i32x4{0, 0, 0, 0};
    // the scales of the columns of gate and up (wave 0) and of the rows (wave 1), on their
    // way into LDS from here
    constexpr int COLS = 16 * CT;
    static_assert(2 * COLS <= 64 && W > 1, "a lane each");
    const float *const mine = w == 0 ? (lane < COLS ? A.gate_scales : A.up_scales) + (int64_t)e * A.inter +
                                           min(tile0 * kI8Cols + lane % COLS, A.inter - 1)
                                     : A.x_scales + slots[min(base + lane, count - 1)] / (uint32_t)A.top_k;
    if (w < 2)
        __builtin_amdgcn_global_load_lds(mine, (__attribute__((address_space(3))) void *)(scales + 64 * w), 4, 0, 0);
    stream<2 * CT, MT, MT == 1 ? 4 : 2>(wt, xr, A.hidden, w, W, steps, acc);
    __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));          // vmcnt(0): they are there
    lane = threadIdx.x;
    asm volatile("" : "+v"(lane));          // addresses are computed here, not held through the products
    lane &= 63, c = lane & 15, j = lane >> 4;
#pragma unroll
    for (int t = 0; t < 2 * CT; ++t)
#pragma unroll
        for (int i = 0; i < MT; ++i) part[w][t * MT + i][lane] = acc[t][i];
    __syncthreads();
    // a wave per column tile and row tile
    const int t = w / MT, i = w % MT, col = (tile0 + t) * kI8Cols + 4 * j;
    if (t < CT && base + 16 * i < count && col < (int)A.ldh) {
        i32x4 a = part[0][2 * t * MT + i][lane], b = part[0][(2 * t + 1) * MT + i][lane];
#pragma unroll
        for (int q = 1; q < W; ++q) a += part[q][2 * t * MT + i][lane], b += part[q][(2 * t + 1) * MT + i][lane];
        const int at = base + 16 * i + c, slot = slots[min(at, count - 1)];
        const float xs = scales[64 + 16 * i + c], *const gs = scales + 16 * t + 4 * j, *const us = gs + COLS;
        float h[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            h[q] = col + q < A.inter ? silu((float)a[q] * xs * gs[q]) * ((float)b[q] * xs * us[q]) : 0.f;
        float *p = A.h + (int64_t)slot * A.ldh + col;
        if constexpr (INSIDE) {
            if (at < count) *(f4 *)p = f4{h[0], h[1], h[2], h[3]};
        } else {
            uint32_t top = max(max(magnitude(h[0]), magnitude(h[1])), max(magnitude(h[2]), magnitude(h[3])));
            top = max(top, (uint32_t)__shfl_xor((int)top, 16));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32));
            if (at < count) {
                share(p, h[0], h[1]);
                share(p + 2, h[2], h[3]);
                if (j == 0)
                    __hip_atomic_store(A.top + (int64_t)slot * tiles + tile0 + t, top, __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
            }
        }
    }
    __syncthreads();
}

// CT: tiles of 16 columns of a workgroup; W: its waves.
template <int CT, int W, bool INSIDE>
__global__ __launch_bounds__(64 * W, 4) void moe_up_kernel(const MoeArgs A) {
    __shared__ uint16_t slots[kMoeMaxSlots];
    __shared__ i32x4 part[W][2 * CT * 2][64];
    __shared__ float scales[128];
    const int all = A.m * A.top_k, tiles = (int)i8_tiles(A.inter), tile0 = blockIdx.x * CT;
    // blockIdx.y: an expert, or where there are fewer slots than experts, a slot, whose
    // expert is taken by the first one that names it
    const bool by_slot = all < A.experts;
    const int e = by_slot ? A.ids[blockIdx.y] : (int)blockIdx.y;
    if ((uint32_t)e >= (uint32_t)A.experts) return;
    const int count = slots_of(A.ids, e, 0, all, slots);
    if (count == 0 || (by_slot && slots[0] != blockIdx.y)) return;
    for (int base = 0; base < count; base += 32) {
        if (count - base <= 16)
            up_rows<CT, 1, W, INSIDE>(A, slots, count, base, e, tile0, tiles, part, scales);
        else
            up_rows<CT, 2, W, INSIDE>(A, slots, count, base, e, tile0, tiles, part, scales);
    }
    if constexpr (INSIDE) return;
    if (!last_to_arrive(A.ctr + e, gridDim.x)) return;
    // this expert's h is whole: 32 rows at a time, the largest magnitude of each from its
    // tiles', then the codes
    __shared__ Step8 st[32];
    const int quads = (int)A.ldh / 4, w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (int base = 0; base < count; base += 32) {
        const int rows = min(32, count - base), work = rows * quads;
        for (int r = w; r < rows; r += W) {
            const int slot = slots[base + r];
            uint32_t top = 0;
            for (int i = lane; i < tiles; i += 64)
                top = max(top, __hip_atomic_load(A.top + (int64_t)slot * tiles + i, __ATOMIC_RELAXED,
                                                 __HIP_MEMORY_SCOPE_AGENT));
            st[r] = step8(wave_max(top));
            if (lane == 0) A.h_scales[slot] = st[r].scale;
        }
        __syncthreads();
        constexpr int U = 4;
        for (int i0 = threadIdx.x; i0 < work; i0 += 64 * W * U) {
            float2 a[U], b[U];
            int64_t at[U];
            int row[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = min(i0 + 64 * W * u, work - 1);
                row[u] = i / quads;
                at[u] = (int64_t)slots[base + row[u]] * A.ldh + 4 * (i - row[u] * quads);
                a[u] = shared2(A.h + at[u]);
                b[u] = shared2(A.h + at[u] + 2);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)            // past the end the last one again: the same bytes
                *(uint32_t *)(A.h8 + at[u]) = codes8(a[u].x, a[u].y, b[u].x, b[u].y, st[row[u]]);
        }
        __syncthreads();
    }
}

// 16 columns of y, by the `parts` workgroups of blockIdx.y together: each takes every
// so-many-th piece of work (an expert and a part of K); the last to arrive adds the
// others' whole-number sums.
constexpr int kDownChunk = 8;       // most fragments of a piece of work
typedef int32_t Sums[16];

// The n slots' sums of all parts; false for a workgroup that is not the last.
__device__ __forceinline__ bool join_parts(const MoeArgs &A, Sums *sums, int n) {
    const int tile = blockIdx.x, parts = gridDim.y;
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));             // addresses are computed here, not held through the products
    if (parts == 1) return true;
    int32_t *const p = A.part + (int64_t)tile * parts * n * 16;
    for (int i = t; i < n * 8; i += 64 * kDownWaves)
        share(p + (int64_t)blockIdx.y * n * 16 + 2 * i, sums[0][2 * i], sums[0][2 * i + 1]);
    if (!last_to_arrive(A.down_ctr + tile, parts)) return false;
    for (int i = t; i < n * 8; i += 64 * kDownWaves) {
        int2 v = make_int2(sums[0][2 * i], sums[0][2 * i + 1]);
        for (int o = 0; o < parts; ++o)
            if (o != (int)blockIdx.y) {
                const int2 u = shared2(p + (int64_t)o * n * 16 + 2 * i);
                v.x += u.x;
                v.y += u.y;
            }
        sums[0][2 * i] = v.x;
        sums[0][2 * i + 1] = v.y;
    }
    __syncthreads();
    return true;
}

// Rows i0 .. of y from their n slots' sums, all slots' scales in one go: sums become
// values, weights those of the slots in use.  d: the scale of this thread's first value,
// if it is loaded already.
template <bool BF16, bool LOADED>
__device__ __forceinline__ void add_slots(const MoeArgs &A, Sums *sums, const int32_t *ids, float *weights,
                                          const float *scales, int i0, int n, float d) {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));             // as above
    for (int i = t; i < n * 16; i += 64 * kDownWaves) {
        const int slot = i / 16, id = ids[slot], col = blockIdx.x * kI8Cols + (i & 15);
        float p = id == -1 ? 0.f : __uint_as_float(0x7fc00000u);
        if ((uint32_t)id < (uint32_t)A.experts && col < A.hidden)
            p = (float)sums[0][i] * scales[slot] * (LOADED ? d : A.down_scales[(int64_t)id * A.hidden + col]);
        sums[0][i] = __float_as_int(p);
    }
    if (t < n) weights[t] = ids[t] == -1 ? 0.f : A.weights[(int64_t)i0 * A.top_k + t];
    __syncthreads();
    for (int i = t; i < n / A.top_k * 16; i += 64 * kDownWaves) {
        const int row = i / 16, col = blockIdx.x * kI8Cols + (i & 15), slot = row * A.top_k;
        if (col >= A.hidden) continue;
        float y = 0.f;
        for (int q = 0; q < A.top_k; ++q) y += weights[slot + q] * __int_as_float(sums[slot + q][i & 15]);
        const int64_t at = (int64_t)(i0 + row) * A.ldy + col;
        if constexpr (BF16)
            ((uint16_t *)A.y)[at] = to_bf16(y);
        else
            ((float *)A.y)[at] = y;
    }
}

// Slots go by groups of whole tokens that LDS has sums for (parts = 1 where that takes
// more than one).
template <bool BF16>
__global__ __launch_bounds__(64 * kDownWaves) void moe_down_kernel(const MoeArgs A) {
    __shared__ Sums sums[kMoeGroup];
    __shared__ int32_t ids[kMoeGroup];
    __shared__ int32_t first[kMoeMaxExperts];      // the first slot of the group that chose an expert
    __shared__ float weights[kMoeGroup];
    __shared__ uint16_t chosen[kMoeGroup];
    __shared__ uint16_t lists[kDownWaves][kMoeGroup];
    const int t = threadIdx.x, lane = t & 63, c = lane & 15, j = lane >> 4, tile = blockIdx.x, parts = gridDim.y;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int steps = (int)i8_steps(A.inter), tiles = gridDim.x, chunks = (steps + kDownChunk - 1) / kDownChunk;
    const int each = (steps + chunks - 1) / chunks;
    const int tokens = min(A.m, kMoeGroup / A.top_k);
    for (int i0 = 0; i0 < A.m; i0 += tokens) {
        const int lo = i0 * A.top_k, n = (min(i0 + tokens, A.m) - i0) * A.top_k;
        for (int i = t; i < A.experts; i += 64 * kDownWaves) first[i] = kMoeGroup;
        __syncthreads();
        for (int i = t; i < n; i += 64 * kDownWaves) {
            const int32_t e = A.ids[lo + i];
            ids[i] = e;
            if ((uint32_t)e < (uint32_t)A.experts) atomicMin(&first[e], i);
        }
        for (int i = t; i < n * 16; i += 64 * kDownWaves) sums[0][i] = 0;
        __syncthreads();
        int active = 0;                            // the chosen experts, listed alike by every wave and part
        for (int k0 = 0; k0 < n; k0 += 64) {
            const int i = k0 + lane;
            const uint32_t e = i < n ? (uint32_t)ids[i] : 0xffffffffu;
            const bool names = e < (uint32_t)A.experts && first[e] == i;
            const uint64_t all = __ballot(names);
            if (names) chosen[active + __popcll(all & ((1ull << lane) - 1))] = (uint16_t)e;
            active += __popcll(all);
        }
        __syncthreads();
        for (int item = w * parts + blockIdx.y; item < active * chunks; item += kDownWaves * parts) {
            const int chunk = item / active, e = chosen[item - chunk * active];
            const int s0 = chunk * each, end = min(s0 + each, steps);
            const char *const wt[1] = {A.down + ((int64_t)e * tiles + tile) * steps * kI8Frag};
            const int count = slots_of(ids, e, 0, n, lists[w]);
            for (int base = 0; base < count; base += 16) {
                const int at = base + c, slot = lists[w][min(at, count - 1)];
                const int8_t *const xr[1] = {A.h8 + (int64_t)(lo + slot) * A.ldh};
                i32x4 acc[1][1] = {{i32x4{0, 0, 0, 0}}};
                stream<1, 1, 8>(wt, xr, (int)A.ldh, s0, 1, end, acc);
                if (at < count)
#pragma unroll
                    for (int q = 0; q < 4; ++q) atomicAdd(&sums[slot][4 * j + q], acc[0][0][q]);
            }
        }
        __syncthreads();
        if (!join_parts(A, sums, n)) return;
        add_slots<BF16, false>(A, sums, ids, weights, A.h_scales + lo, i0, n, 0.f);
        __syncthreads();
    }
}

// Up to 16 slots of short rows: a wave turns a row of h into codes while its
// first piece of the weights is on its way, and finds the pieces of work from the ids
// in its registers.
constexpr int kHeld = 4;            // quads of a row of h that a lane holds
template <bool BF16>
__global__ __launch_bounds__(64 * kDownWaves) void moe_down_few_kernel(const MoeArgs A) {
    __shared__ __attribute__((aligned(16))) int8_t codes[kDownWaves * (kMoeInside + 16)];
    __shared__ float scales[kDownWaves];
    __shared__ Sums sums[kDownWaves];
    __shared__ int32_t ids[kDownWaves];
    __shared__ float weights[kDownWaves];
    const int t = threadIdx.x, lane = t & 63, c = lane & 15, j = lane >> 4, tile = blockIdx.x, parts = gridDim.y;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6), n = A.m * A.top_k;
    const int steps = (int)i8_steps(A.inter), tiles = gridDim.x, chunks = (steps + kDownChunk - 1) / kDownChunk;
    const int each = (steps + chunks - 1) / chunks;
    const int stride = (int)A.ldh + 16, quads = (int)A.ldh / 4;          // rows of codes, 16 of them in different banks
    const int id = lane < n ? A.ids[lane] : -1, own = t < 16 * n ? A.ids[t / 16] : -1;
    const f4 *const row = (const f4 *)(A.h + (int64_t)min(w, n - 1) * A.ldh);
    f4 v[kHeld];
#pragma unroll
    for (int q = 0; q < kHeld; ++q) v[q] = row[min(64 * q + lane, quads - 1)];
    __builtin_amdgcn_sched_barrier(0);
    bool first = (uint32_t)id < (uint32_t)A.experts;       // no lane before has the same expert
#pragma unroll
    for (int q = 0; q < kDownWaves - 1; ++q) first &= (lane <= q) | (__builtin_amdgcn_readlane(id, q) != id);
    const uint64_t experts = __ballot(first);
    const int active = __popcll(experts), rank = __popcll(experts & ((1ull << lane) - 1));
    const int all = active * chunks, by = kDownWaves * parts;
    i32x4 f[kDownChunk];
    int item = w * parts + blockIdx.y, e = 0, s0 = 0, end = 0;
    const auto fetch = [&]() __attribute__((always_inline)) {
        const int chunk = item / active, at = item - chunk * active;
        e = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)__ballot(first && rank == at)) - 1);
        s0 = chunk * each, end = min(s0 + each, steps);
        const char *const wt = A.down + ((int64_t)e * tiles + tile) * steps * kI8Frag + 16 * lane;
#pragma unroll
        for (int u = 0; u < kDownChunk; ++u)
            f[u] = __builtin_nontemporal_load((const i32x4 *)(wt + (int64_t)min(s0 + u, end - 1) * kI8Frag));
        __builtin_amdgcn_sched_barrier(0);
    };
    if (item < all) fetch();
    // the scale of this thread's slot and column
    const int col = tile * kI8Cols + (t & 15);
    const float d = (uint32_t)own < (uint32_t)A.experts && col < A.hidden ? A.down_scales[(int64_t)own * A.hidden + col] : 0.f;
    if (w == 0 && lane < n) ids[lane] = id;
    if (t < 16 * kDownWaves) sums[0][t] = 0;
    if (w < n) {
        uint32_t top = 0;
        const auto most = [&](const f4 &x) {
            top = max(top, max(max(magnitude(x[0]), magnitude(x[1])), max(magnitude(x[2]), magnitude(x[3]))));
        };
#pragma unroll
        for (int q = 0; q < kHeld; ++q) most(v[q]);
        for (int q = 64 * kHeld + lane; q < quads; q += 64) most(row[q]);
        const Step8 st = step8(wave_max(top));
        uint32_t *const out = (uint32_t *)(codes + w * stride);
#pragma unroll
        for (int q = 0; q < kHeld; ++q)
            if (64 * q + lane < quads) out[64 * q + lane] = codes8(v[q][0], v[q][1], v[q][2], v[q][3], st);
        for (int q = 64 * kHeld + lane; q < quads; q += 64) {
            const f4 x = row[q];
            out[q] = codes8(x[0], x[1], x[2], x[3], st);
        }
        if (lane == 0) scales[w] = st.scale;
    }
    __syncthreads();
    while (item < all) {
        // column c of the product is the c-th slot that chose e
        const uint64_t mine = __ballot(id == e);
        const int count = __popcll(mine);
        int slot = 0, seen = 0;
#pragma unroll
        for (int q = 0; q < kDownWaves; ++q)
            if (mine >> q & 1) {
                slot = seen == c ? q : slot;
                ++seen;
            }
        const int8_t *const x = codes + slot * stride + 16 * j;
        i32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < kDownChunk; ++u) {
            const int r = (s0 + u) * kI8K;                 // past ldh, where the weights are zeros, the first codes
            if (s0 + u < end) acc = mfma64(f[u], *(const i32x4 *)(x + (r + 16 * j < (int)A.ldh ? r : 0)), acc);
        }
        item += by;
        if (item < all) fetch();
        if (c < count)
#pragma unroll
            for (int q = 0; q < 4; ++q) atomicAdd(&sums[slot][4 * j + q], acc[q]);
    }
    __syncthreads();
    if (!join_parts(A, sums, n)) return;
    add_slots<BF16, true>(A, sums, ids, weights, scales, 0, n, d);
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs &a, hipStream_t s) {
    // A workgroup per row against one per 16 experts, 1 / 8 / 64 rows (us): 8 experts of 2048
    // 5.8 / 6.1 / 6.3 against 4.8 / 5.8 / 15.5, of 4096 5.8 / 6.1 / 6.3 against 6.3 / 8.0 / 23.6; 16 of 4096
    // 7.0 / 7.4 / 7.5 against 7.7 / 9.1 / 24.7; 32 of 2048 7.0 / 7.2 / 7.4 against 5.7 / 6.6 / 16.6; 64 of
    // 4096 19.8 / 20.2 / 20.2 against 7.9 / 9.3 / 25.2; 128 of 2048 19.8 / 20.2 / 20.2 against
    // 6.0 / 7.0 / 17.7.  One bound for all row counts, so some us are left at either side of it.
    const dim3 grid((a.experts + 15) / 16), block(64 * kRouteWaves);
    if ((int64_t)a.experts * a.k <= 48 << 10)
        hipLaunchKernelGGL(route_row_kernel, dim3(a.m), block, 0, s, a);
    else if (a.m <= 16)
        hipLaunchKernelGGL((route_kernel<1>), grid, block, 0, s, a);
    else if (a.m <= 32)
        hipLaunchKernelGGL((route_kernel<2>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((route_kernel<4>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <bool INSIDE>
hipError_t launch_inside(const MoeArgs &a, hipStream_t s) {
    const int slots = a.m * a.top_k, most = slots < a.experts ? slots : a.experts;
    // 32 columns of gate and up per workgroup; its waves take 8 fragments or more each
    // (with h's codes made here, 1 / 6 rows of 8 of 128 experts 2048 -> 768, 32 rows of 2 of
    // 8 4096 -> 14336: four waves 9.5 / 27.4 / 179 us, eight 9.8 / 30.0 / 173; 16 columns and
    // four 10.1 / 29.4 / 193)
    const dim3 up((unsigned)((i8_tiles(a.inter) + 1) / 2), most);
    if (i8_steps(a.hidden) >= 48)
        hipLaunchKernelGGL((moe_up_kernel<2, 8, INSIDE>), up, dim3(512), 0, s, a);
    else
        hipLaunchKernelGGL((moe_up_kernel<2, 4, INSIDE>), up, dim3(256), 0, s, a);
    const dim3 down((unsigned)i8_tiles(a.hidden), a.parts), block(64 * kDownWaves);
    if (INSIDE && a.y_bf16)
        hipLaunchKernelGGL((moe_down_few_kernel<true>), down, block, 0, s, a);
    else if (INSIDE)
        hipLaunchKernelGGL((moe_down_few_kernel<false>), down, block, 0, s, a);
    else if (a.y_bf16)
        hipLaunchKernelGGL((moe_down_kernel<true>), down, block, 0, s, a);
    else
        hipLaunchKernelGGL((moe_down_kernel<false>), down, block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_moe_mlp(const MoeArgs &a, hipStream_t s) {
    return a.inside ? launch_inside<true>(a, s) : launch_inside<false>(a, s);
}

}  // namespace dspk
