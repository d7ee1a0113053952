// Products of 8-bit rows with 8-bit weights, and the weights' packing:
//   y[i][c] = float(sum_r x[i][r] w[c][r]) * x_scales[i] * w_scales[c]
// with 16x16x64 integer matrix instructions.  The sums are exact, so kernels, splits
// and orders of K all give the same bits; i8_plan chooses among them by time alone.
//
// Few rows (streams) are bound by the weight's way from memory: 19456x2560 over one
// row 9.1-9.8 us (5.1-5.5 TB/s), 40960x2560 16.7 (6.3), 5120x17408 15.9 (5.6); a large
// copy moves 5.1 TB/s on this card.  Many rows (tiles) are bound by the matrix units'
// power: with every operand in registers random codes reach 3.96 POP/s (zeros 4.8), with
// operands from LDS 3.3, the kernel 2.4 (8192^3, 455 us).  32x32x32 instructions
// need more of it: 3.3 POP/s from registers, 2.9 from LDS, 2.2 in the kernel.  In between
// the caches' rate to the CUs (some 16 TB/s) decides: it is why 301 rows of 6144x4096
// take 15.7 us, with weights and rows read again by every tile.
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

// -------------------------------------------------------------------- few rows
// A workgroup takes CT tiles of 16 columns and up to 16 MT rows over the whole of K.
// Wave w of W streams fragments w, w + W, .. of each tile, and the same pieces of x,
// through a ring of D register sets; the waves' sums meet in LDS.  The weight is the
// instruction's first operand, so that a lane ends with four neighbouring columns of
// one row.
template <int MT, int CT, int D, bool BF16>
__global__ __launch_bounds__(1024, 4) void i8_stream_kernel(const I8GemmArgs A) {
    extern __shared__ i32x4 part[];                // [wave][CT][MT][lane]
    const int lane = threadIdx.x & 63, c = lane & 15, j = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int tile0 = blockIdx.x * CT;
    const char *wt[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t) wt[t] = A.tiles + (int64_t)min(tile0 + t, A.tiles_n - 1) * A.steps * kI8Frag;
    const char *const xb = (const char *)A.x;
    uint32_t xo[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) xo[i] = (uint32_t)min(16 * i + c, A.m - 1) * (uint32_t)A.ldx;
    struct Set {
        i32x4 f[CT], x[MT];
    };
    // fragment s; past the last one that one again, as zeros
    auto load = [&](int s, Set &o) __attribute__((always_inline)) {
        const int at = min(s, A.steps - 1);
#pragma unroll
        for (int t = 0; t < CT; ++t)
            o.f[t] = __builtin_nontemporal_load((const i32x4 *)(wt[t] + (int64_t)at * kI8Frag + 16 * lane));
        const uint32_t r = (uint32_t)at * kI8K + 16 * j, in = r < (uint32_t)A.k ? r : 0u;       // past k: meets zeros
#pragma unroll
        for (int i = 0; i < MT; ++i) o.x[i] = *(const i32x4 *)(xb + (xo[i] + in));
    };
    i32x4 acc[CT][MT];
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[t][i] = i32x4{0, 0, 0, 0};
    auto multiply = [&](int s, const Set &o) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            const i32x4 f = s < A.steps ? o.f[t] : i32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[t][i] = mfma64(f, o.x[i], acc[t][i]);
        }
    };
    Set ring[D];
    int s0 = w;
#pragma unroll
    for (int u = 0; u < D; ++u) load(s0 + u * waves, ring[u]);
    __builtin_amdgcn_sched_barrier(0);
    for (; s0 + D * waves < A.steps; s0 += D * waves) {
#pragma unroll
        for (int u = 0; u < D; ++u) {
            multiply(s0 + u * waves, ring[u]);
            load(s0 + (D + u) * waves, ring[u]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int u = 0; u < D; ++u) multiply(s0 + u * waves, ring[u]);

    // each thread's four columns of a row; their scales on their way while the sums meet
    int row, col;
    float xs, ws[4];
    auto take = [&](int q) __attribute__((always_inline)) {
        row = 16 * ((q >> 6) % MT) + (q & 15);
        col = (tile0 + (q >> 6) / MT) * kI8Cols + 4 * ((q >> 4) & 3);
        xs = A.x_scales[min(row, A.m - 1)];
#pragma unroll
        for (int e = 0; e < 4; ++e) ws[e] = A.w_scales[min(col + e, A.n - 1)];
    };
    take(threadIdx.x);
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int i = 0; i < MT; ++i) part[((w * CT + t) * MT + i) * 64 + lane] = acc[t][i];
    __syncthreads();
    for (int q = threadIdx.x; q < CT * MT * 64; q += blockDim.x) {
        if (q != (int)threadIdx.x) take(q);
        i32x4 sum = part[q];
        for (int i = 1; i < waves; ++i) sum += part[i * CT * MT * 64 + q];
        if (row >= A.m || col >= A.n) continue;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)sum[e] * xs * ws[e];
        store4<BF16>(A.y, row * A.ldy + col, col, A.n, A.vec, v);
    }
}

template <int MT, int CT, int D>
hipError_t launch_stream(const I8GemmArgs &a, const I8Plan &p, hipStream_t s) {
    const dim3 grid((unsigned)p.groups), block(64 * p.waves);
    const size_t lds = (size_t)p.waves * MT * CT * 1024;
    if (a.y_bf16)
        hipLaunchKernelGGL((i8_stream_kernel<MT, CT, D, true>), grid, block, lds, s, a);
    else
        hipLaunchKernelGGL((i8_stream_kernel<MT, CT, D, false>), grid, block, lds, s, a);
    return hipGetLastError();
}

// ------------------------------------------------------------------- many rows
// A workgroup of WR x WC waves takes BM rows x BN columns, a wave 16 TX rows x 16 TW
// columns of it.  K goes by stages of KS through a ring of NB buffers in LDS, filled by
// direct global-to-LDS loads NB - 1 stages ahead.
// Rows of x lie KS bytes apart, 16-byte piece p of row r at a place of its line that
// depends on r, so that 16 neighbouring rows' pieces, which an LDS cycle reads, are
// in different banks; weight fragments lie as in memory.
// Eight waves take 16 or 32 rows x 32 columns each (64 x 32 of a 128 x 128 tile; a 32 x 64
// tile has four of 32 x 16): with four waves of 32 x 64 the 64 x 128 tiles take 19.1 us
// instead of 16.6 (301 rows of 6144x4096); 64 x 64 tiles with five buffers, of which one
// workgroup fits a CU, 24.1 instead of 14.9 (320 of 4096x4096).  Deeper rings and 256 K per
// stage are slower.
constexpr int KS = 128;
template <int WR, int WC, int TX, int TW, int NB>
struct Tile {
    static constexpr int WAVES = WR * WC, BM = 16 * WR * TX, BN = 16 * WC * TW;
    static constexpr int XB = BM * KS, WB = BN * KS, STAGE = XB + WB;       // bytes of a stage
    static constexpr int XI = XB / 1024 / WAVES, WI = WB / 1024 / WAVES;    // loads of a wave
    static_assert(XI * WAVES * 1024 == XB && WI * WAVES * 1024 == WB, "loads split evenly over the waves");
    static_assert(NB * STAGE <= 160 * 1024, "LDS");
    static constexpr int P = KS / 16, R = 64 / P;      // pieces of a row, rows of a load
    // the line of row r and the place of its piece p
    static __device__ __forceinline__ int line(int r) { return r ^ (r >> 3 & 1); }
    static __device__ __forceinline__ int place(int r, int p) { return p ^ (r & 7); }
};

__device__ __forceinline__ void to_lds(const void *src, char *dst) {
    __builtin_amdgcn_global_load_lds(src, (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
}
// This wave's loads but the last N have arrived, its LDS reads too; then all waves are here.
template <int N>
__device__ __forceinline__ void arrive() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (N >> 4) << 14);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// One run of the numbers 0 .. all - 1 for each of the eight dies, which workgroups go
// to in turn: what a die runs at a time is neighbouring and shares its cache.
constexpr int kDies = 8;
__device__ __forceinline__ int on_die(int i, int all) {
    const int die = i % kDies;
    return die * (all / kDies) + min(die, all % kDies) + i / kDies;
}
// Tile `at` of rows x cols: kBand row tiles down, then the next column.
constexpr int kBand = 4;
__device__ __forceinline__ void tile_of(int at, int rows, int cols, int &r, int &c) {
    const int band = at / (kBand * cols), high = min(kBand, rows - band * kBand), in = at - band * kBand * cols;
    c = in / high;
    r = band * kBand + in - c * high;
}

// A stage's buffers.
struct Buffers {
    char *x, *w;
};

// The tile at row0 and 16-column tile tile0, over a ring of NB buffers.
// SPLIT: workgroup blockIdx.y of A.splits takes its part of K; the last of them to
// arrive adds the others' sums (whole numbers: in any order the same).
template <int WR, int WC, int TX, int TW, int NB, bool SPLIT, bool BF16>
__device__ __forceinline__ void tile_work(const I8GemmArgs &A, int row0, int tile0, const Buffers (&ring)[NB]) {
    using T = Tile<WR, WC, TX, TW, NB>;
    static_assert(NB >= 2 && NB <= 4, "ring");
    constexpr int L = T::XI + T::WI;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = w / WC, wc = w % WC;
    i32x4 acc[TX][TW];
#pragma unroll
    for (int i = 0; i < TX; ++i)
#pragma unroll
        for (int t = 0; t < TW; ++t) acc[i][t] = i32x4{0, 0, 0, 0};

    // Stage s into a buffer.  Rows past m read the last one, tiles past n the last one;
    // K past k: x reads column 0, which meets the zeros of the weight.  A lane's part of
    // an address stays the same from stage to stage, the uniform part moves.
    const char *const xb = (const char *)A.x + (int64_t)row0 * A.ldx;
    uint32_t xo[T::XI];
    int col[T::XI];
    const char *wq[T::WI];
#pragma unroll
    for (int q = 0; q < T::XI; ++q) {
        const int r = T::line(T::R * (w * T::XI + q) + lane / T::P);
        col[q] = 16 * T::place(r, lane % T::P);
        xo[q] = (uint32_t)min(r, A.m - 1 - row0) * (uint32_t)A.ldx + col[q];
    }
#pragma unroll
    for (int q = 0; q < T::WI; ++q) {
        constexpr int F = KS / kI8K;               // fragments of a tile and stage
        const int i = w * T::WI + q;
        wq[q] = A.tiles + ((int64_t)min(tile0 + i / F, A.tiles_n - 1) * A.steps + i % F) * kI8Frag;
    }
    int first = 0, stages = A.steps * kI8K / KS;   // this workgroup's stages [first, stages)
    if constexpr (SPLIT) {
        const int all = stages;
        first = (int)((int64_t)all * blockIdx.y / A.splits);
        stages = (int)((int64_t)all * (blockIdx.y + 1) / A.splits);
    }
    auto fill = [&](int s, const Buffers &to) __attribute__((always_inline)) {
        const uint32_t at = (uint32_t)s * KS;
#pragma unroll
        for (int q = 0; q < T::XI; ++q)
            to_lds(xb + (xo[q] + (at + col[q] < (uint32_t)A.k ? at : 0u - col[q])), to.x + 1024 * (w * T::XI + q));
#pragma unroll
        for (int q = 0; q < T::WI; ++q)
            to_lds(wq[q] + (uint64_t)s * (KS * kI8Cols) + 16 * lane, to.w + 1024 * (w * T::WI + q));
    };
    const int xrow = 16 * TX * wr + (lane & 15), j = lane >> 4;
    const int wat = TW * wc * (KS * kI8Cols) + 16 * lane;
    // Lane l ends with row l % 16 and columns 4 (l / 16) .. + 3 of each 16 x 16 product.
    // Their scales: small waves' at once, where the registers hold them.
    constexpr bool EARLY = TX * TW <= 4;
    float xs[TX], ws[TW][4];
    auto scales = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < TX; ++i) xs[i] = A.x_scales[min(row0 + xrow + 16 * i, A.m - 1)];
#pragma unroll
        for (int t = 0; t < TW; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                ws[t][e] = A.w_scales[min((tile0 + TW * wc + t) * kI8Cols + 4 * j + e, A.n - 1)];
    };
    if constexpr (EARLY) scales();
    struct Operands {
        i32x4 a[TW], b[TX];
    };
    auto read = [&](const Buffers &from, int h, Operands &o) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < TW; ++t) o.a[t] = *(const i32x4 *)(from.w + wat + KS * kI8Cols * t + kI8Frag * h);
#pragma unroll
        for (int i = 0; i < TX; ++i)
            o.b[i] = *(const i32x4 *)(from.x + (T::line(xrow) + 16 * i) * KS + 16 * T::place(xrow, 4 * h + j));
    };
    // A stage's steps of 64 K, each step's operands read while the one before is
    // multiplied, and the stage NB - 1 further on started on its way to the buffer that
    // was read last.
    auto stage = [&](int s, const Buffers &from, const Buffers &next) __attribute__((always_inline)) {
        if (s + NB - 2 < stages)
            arrive<(NB - 2) * L>();
        else
            arrive<0>();
        Operands o[2];
        read(from, 0, o[0]);
        if (s + NB - 1 < stages) fill(s + NB - 1, next);
#pragma unroll
        for (int h = 0; h < KS / 64; ++h) {
            if (h + 1 < KS / 64) read(from, h + 1, o[(h + 1) & 1]);
#pragma unroll
            for (int i = 0; i < TX; ++i)
#pragma unroll
                for (int t = 0; t < TW; ++t) acc[i][t] = mfma64(o[h & 1].a[t], o[h & 1].b[i], acc[i][t]);
            // a read after each two of the first products: the next step's operands
            // arrive while these are under way
            if constexpr (TX * TW > 2 * (TX + TW))
                if (h + 1 < KS / 64)
#pragma unroll
                    for (int e = 0; e < TX + TW; ++e) {
                        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
                        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                    }
        }
    };
#pragma unroll
    for (int s = 0; s < NB - 1; ++s)
        if (first + s < stages) fill(first + s, ring[s]);
    for (int s0 = first; s0 < stages; s0 += NB) {
#pragma unroll
        for (int u = 0; u < NB; ++u)
            if (s0 + u < stages) stage(s0 + u, ring[u], ring[(u + NB - 1) % NB]);
    }
    if constexpr (SPLIT)
        if (A.splits > 1) {
            constexpr int PW = TX * TW * 256;      // sums of a wave
            int32_t *const p = A.part + ((int64_t)blockIdx.x * A.splits * T::WAVES + w) * PW + 2 * lane;
#pragma unroll
            for (int i = 0; i < TX; ++i)
#pragma unroll
                for (int t = 0; t < TW; ++t) {
                    int32_t *const q = p + (int64_t)blockIdx.y * T::WAVES * PW + (i * TW + t) * 256;
                    share(q, acc[i][t][0], acc[i][t][1]);
                    share(q + 128, acc[i][t][2], acc[i][t][3]);
                }
            if (!last_to_arrive(A.ctr + blockIdx.x, A.splits)) return;
            for (int o = 0; o < A.splits; ++o) {
                if (o == (int)blockIdx.y) continue;
#pragma unroll
                for (int i = 0; i < TX; ++i)
#pragma unroll
                    for (int t = 0; t < TW; ++t) {
                        const int32_t *const q = p + (int64_t)o * T::WAVES * PW + (i * TW + t) * 256;
                        const int2 lo = shared2(q), hi = shared2(q + 128);
                        acc[i][t] += i32x4{lo.x, lo.y, hi.x, hi.y};
                    }
            }
        }
    if constexpr (!EARLY) scales();
#pragma unroll
    for (int t = 0; t < TW; ++t) {
        const int c = (tile0 + TW * wc + t) * kI8Cols + 4 * j;
        if (c >= A.n) continue;
#pragma unroll
        for (int i = 0; i < TX; ++i) {
            const int row = row0 + xrow + 16 * i;
            if (row >= A.m) continue;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][t][e] * xs[i] * ws[t][e];
            store4<BF16>(A.y, row * A.ldy + c, c, A.n, A.vec, v);
        }
    }
}

template <int WR, int WC, int TX, int TW, int NB, int OCC, bool BF16>
__global__ __launch_bounds__(64 * WR * WC, OCC) void i8_tile_kernel(const I8GemmArgs A) {
    using T = Tile<WR, WC, TX, TW, NB>;
    __shared__ __attribute__((aligned(1024))) char b0[T::STAGE], b1[T::STAGE], b2[NB > 2 ? T::STAGE : 16],
        b3[NB > 3 ? T::STAGE : 16];
    char *const every[4] = {b0, b1, b2, b3};
    Buffers ring[NB];
#pragma unroll
    for (int u = 0; u < NB; ++u) ring[u] = {every[u], every[u] + T::XB};
    const int rows = (A.m + T::BM - 1) / T::BM, cols = (A.n + T::BN - 1) / T::BN;
    int r, c;
    tile_of(on_die(blockIdx.x, rows * cols), rows, cols, r, c);
    tile_work<WR, WC, TX, TW, NB, true, BF16>(A, r * T::BM, c * (T::BN / kI8Cols), ring);
}

template <int WR, int WC, int TX, int TW, int NB, int OCC>
hipError_t launch_tile(const I8GemmArgs &a, const I8Plan &p, hipStream_t s) {
    using T = Tile<WR, WC, TX, TW, NB>;
    const dim3 grid((unsigned)p.groups, a.splits), block(64 * T::WAVES);
    if (a.y_bf16)
        hipLaunchKernelGGL((i8_tile_kernel<WR, WC, TX, TW, NB, OCC, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((i8_tile_kernel<WR, WC, TX, TW, NB, OCC, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

// Tiles of 256 x 256, one workgroup per CU; the last of them, where they would leave
// CUs without work, as four of 128 x 128 each (4096 rows of 17408x5120, 1088 tiles:
// 8% less time than without; 334 to 340 us, 2.15 POP/s).  Two buffers of 128 K each: four of 64 measure the same
// (8192^3 470 against 458 us), 128 x 64 wave tiles turned the other way too (463).
template <bool BF16>
__global__ __launch_bounds__(512, 2) void i8_big_kernel(const I8GemmArgs A) {
    using B = Tile<4, 2, 4, 8, 2>;
    using Q = Tile<2, 4, 4, 2, 4>;
    static_assert(B::XB == Q::STAGE && B::WB == Q::STAGE, "a quarter's stage takes half a whole one's");
    __shared__ __attribute__((aligned(1024))) char b0[Q::STAGE], b1[Q::STAGE], b2[Q::STAGE], b3[Q::STAGE];
    const int rows = (A.m + B::BM - 1) / B::BM, cols = (A.n + B::BN - 1) / B::BN, i = blockIdx.x;
    int r, c;
    if (i < A.whole) {
        tile_of(on_die(i, A.whole), rows, cols, r, c);
        tile_work<4, 2, 4, 8, 2, false, BF16>(A, r * B::BM, c * (B::BN / kI8Cols), {{b0, b1}, {b2, b3}});
        return;
    }
    const int at = on_die(i - A.whole, gridDim.x - A.whole);
    tile_of(A.whole + at / 4, rows, cols, r, c);
    const int row0 = r * B::BM + (at & 1) * (B::BM / 2), tile0 = (2 * c + (at >> 1 & 1)) * (B::BN / kI8Cols / 2);
    if (row0 >= A.m || tile0 >= A.tiles_n) return;
    tile_work<2, 4, 4, 2, 4, false, BF16>(
        A, row0, tile0, {{b0, b0 + Q::XB}, {b1, b1 + Q::XB}, {b2, b2 + Q::XB}, {b3, b3 + Q::XB}});
}
hipError_t launch_big(const I8GemmArgs &a, const I8Plan &p, hipStream_t s) {
    const dim3 grid((unsigned)p.groups), block(512);
    if (a.y_bf16)
        hipLaunchKernelGGL((i8_big_kernel<true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((i8_big_kernel<false>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_pack(const I8PackArgs &a, hipStream_t s) {
    const int64_t blocks = (a.tiles * a.steps * 64 + 255) / 256;
    hipLaunchKernelGGL(i8_pack_kernel, dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20)), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_i8_gemm(const I8GemmArgs &a, const I8Plan &p, hipStream_t s) {
    switch (p.kind) {
        case kI8Stream16x1: return launch_stream<1, 1, 8>(a, p, s);
        case kI8Stream16x2: return launch_stream<1, 2, 4>(a, p, s);
        case kI8Stream32x1: return launch_stream<2, 1, 4>(a, p, s);
        case kI8Stream32x2: return launch_stream<2, 2, 4>(a, p, s);
        case kI8Stream64x1: return launch_stream<4, 1, 4>(a, p, s);
        case kI8Stream64x2: return launch_stream<4, 2, 2>(a, p, s);
        case kI8Tile32x64: return launch_tile<1, 4, 2, 1, 4, 2>(a, p, s);
        case kI8Tile64x64: return launch_tile<4, 2, 1, 2, 4, 2>(a, p, s);
        case kI8Tile64x128: return launch_tile<2, 4, 2, 2, 3, 2>(a, p, s);
        case kI8Tile128x128: return launch_tile<2, 4, 4, 2, 2, 2>(a, p, s);
        case kI8Tile256x256: return launch_big(a, p, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace dspk
