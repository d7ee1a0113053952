// Attention of a round's rows over the paged cache: one token, a chain or a
// tree of up to 64 drafts per request, any number of requests, q heads in
// groups over the k/v heads.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i.k_j - max_j),
//
// j over the positions row i sees.  The rows of a request over one kv head are
// cut into blocks of 16 or 32 (what a wave's registers hold; attn_plan says
// which).  A (request, kv head) is a segment, its cache positions are cut into
// units of 256; groups of workgroups, one for each row block, take equal
// contiguous ranges of all segments' units, so ragged batches load every CU
// alike.  A group's workgroups sit on one XCD and stream the same k and v at the
// same time, out of its L2 for all but the first (3 row blocks: 84 MB missed L2
// of 240 MB asked for).  A segment shared by groups leaves partial sums in the
// workspace; the last to arrive adds them in order (deterministic), each wave
// its own tiles, or a launch of its own does where they may be many.  The host,
// which does not know the lengths, plans for those that the page table has room
// for: one token over 1021 positions takes 8.3 us under a table of that size, 12.5
// under one of 8 or 128 times it (a launch of its own that finds little to add).
//
// Within a workgroup each wave takes its own positions, so k and v go from
// memory to the matrix cores without LDS or barriers: the cache is stored in
// operand order (kv_layout.h).  Scores are computed as S^T = K Q^T, whose
// result layout (lane: one row, four neighbouring positions) is already the
// operand layout of O^T = V^T P^T; every statistic of a row lies in its
// lanes, one value each.  The waves' results are joined through LDS when a
// segment ends.
//
// Rounding: scores, statistics, sums and outputs are fp32.  Over a bf16 cache a
// probability goes into the second product as the sum of two bf16 (16
// significant bits): with one the output's error would be 1.4 times that of the
// final rounding alone, and the matrix cores have the time.  8-bit codes are exact in
// bf16 and fp16; their scales multiply scores and probabilities in fp32, and
// the scaled probability goes in as one fp16 (11 bits, 2^-12 at most: a
// hundredth of the output's own rounding in the mean square).
//
// What bounds it, measured on MI355X as passes back to back (32 q heads over 8
// of 128 unless said): one token over 1021 positions 8.2 us, of which 2.2 is the
// launch, 1.5 the lengths' way to the first page number, 1 the only step, 3.5
// the way of the results through LDS, memory and the last workgroup; 4 requests
// of 6 rows over up to 8190 positions 25.7 us (97 MB); 32 of 8 rows over up to
// 16384 (1.37 GB) 248 us, 5.5 TB/s of the 6.5 this device streams.  Over 8-bit
// caches of many rows the vector ALUs: decoding takes half of their work (17 rows
// of 40 heads over 32768 positions, 70 MB: 39 us, ALUs busy for 55% of it), and
// the scores' spread: see the references below.
#include <hip/hip_runtime.h>

#include "decode.h"
#include "kv_layout.h"

namespace dspk {
namespace {

using dec::as_bf16x8;
using dec::bf16x8;
using kv::f32x4;
using kv::u32x4;
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int WAVES = kAttnWaves, TPB = 64 * WAVES;
constexpr int kStep = kAttnStep;        // positions of a wave's step
constexpr int kTileFloats = kAttnTile;  // a tile of partial sums: 16 x 16 outputs, and m and sum of 16 rows
constexpr int kUnit = kAttnStep * WAVES;
constexpr int kJoinWaves = 4;

#define NEG_INF (-__builtin_inff())
// Limits of what a lane adds at a time, in units of its row's reference, before
// the reference has to rise.  8 bits: a probability times its v scale goes into
// the product as fp16, at most 2^15, 2^4 at the reference; it keeps its 11 bits
// down to 2^-18 of the reference; the sum of probabilities alone, which small v
// scales let grow to 2^54 at the reference, has fp32's range.  bf16: products with
// v share that range, of which v has what 2^32 per position leaves, up to 2^78 at
// 2^17 positions.
constexpr float kMostF16 = 32768.f, kBase8 = 4.f;
template <int BITS>
constexpr float kMostSum = BITS == 8 ? 0x1p60f : 0x1p32f;
// The reference of a row that has seen nothing yet, for 2^(-inf - ref) = 0.
__device__ __forceinline__ float zero_if_none(float m) { return m == NEG_INF ? 0.f : m; }

// Byte i of x, signed, as a float: one instruction (the compiler would
// extract, extend and convert).
template <int I>
__device__ __forceinline__ float byte_f32(uint32_t x) {
    float r;
    if constexpr (I == 0)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0" : "=v"(r) : "v"(x));
    else if constexpr (I == 1)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1" : "=v"(r) : "v"(x));
    else if constexpr (I == 2)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2" : "=v"(r) : "v"(x));
    else
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3" : "=v"(r) : "v"(x));
    return r;
}
// Eight signed codes (two dwords, lowest byte first) as exact bf16 values.
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t a, uint32_t b) {
    u32x4 r;
    r[0] = dec::pack_hi16(byte_f32<0>(a), byte_f32<1>(a));
    r[1] = dec::pack_hi16(byte_f32<2>(a), byte_f32<3>(a));
    r[2] = dec::pack_hi16(byte_f32<0>(b), byte_f32<1>(b));
    r[3] = dec::pack_hi16(byte_f32<2>(b), byte_f32<3>(b));
    return as_bf16x8(r);
}

// Eight signed codes as exact fp16 values: u = code + 128 under the exponent of
// 1024 is 1024 + u, less 1152 the code.
__device__ __forceinline__ f16x8 codes_f16(uint32_t a, uint32_t b) {
    const f16x2 off = {(_Float16)-1152.f, (_Float16)-1152.f};
    a ^= 0x80808080u;
    b ^= 0x80808080u;
    u32x4 r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, a, 0x04010400u)) + off);
    r[1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, a, 0x04030402u)) + off);
    r[2] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u)) + off);
    r[3] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u)) + off);
    return __builtin_bit_cast(f16x8, r);
}

// The largest of three, NaN left aside (written out: the compiler would first
// quieten results of the matrix cores).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// max and sum over the four lanes of a row (lane % 16 is the row)
__device__ __forceinline__ float row_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float row_sum(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// Units of a request: per segment and in all.  A request with rows has at
// least one unit per segment, so that its rows are written even if nothing is
// cached or its length is a fault.
struct Units {
    int per_seg, total;
};
__device__ __forceinline__ Units units_of(const AttnArgs &A, const kv::Req &q) {
    Units u;
    u.per_seg = max(1, ((q.ok ? q.len + q.rows : 0) + kUnit - 1) / kUnit);
    u.total = q.rows > 0 ? u.per_seg * A.c.heads : 0;
    return u;
}

// Range of a group: the first rem groups take q + 1 units, the others q.  The
// inverse gives the group of a unit.
struct Ranges {
    int q, rem;
    __device__ __forceinline__ int begin(int w) const { return w * q + min(w, rem); }
    __device__ __forceinline__ int owner(int u) const {
        const int cut = rem * (q + 1);
        return u < cut ? u / (q + 1) : rem + (u - cut) / q;
    }
};
__device__ __forceinline__ Ranges ranges(const AttnArgs &A, int total) {
    // Fewer than two units each: two to some, which is no slower and leaves fewer
    // pieces.  Segments of two: whole, for a second step costs less than a join
    // (one token over 300 to 500 positions 6.5 to 7.5 us, else 8.5).
    const bool two = total < 2 * A.groups && (total > A.groups || A.pairs);
    const int groups = two ? max(1, (total + 1) / 2) : A.groups;
    Ranges R;
    R.q = total / groups;
    R.rem = total - R.q * groups;
    return R;
}

// A group's range, and where it starts: the request that holds its first unit
// and that request's first unit.  Every wave does it by itself; requests are
// taken 64 at a time, one per lane.
struct Start {
    int u, u_end, req, first;
    kv::Req q;
};
__device__ __forceinline__ int prefix_sum(int x) {                  // inclusive, over the lanes
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(x, o);
        if (lane >= o) x += y;
    }
    return x;
}
__device__ __forceinline__ Start find_start(const AttnArgs &A, int group, Ranges &R) {
    const int lane = threadIdx.x & 63;
    int total = 0, x = 0, u = 0;
    kv::Req q = {};
    const auto load = [&](int base) {
        u = 0;
        if (base + lane < A.B.b) {
            q = kv::request(A.B, A.c.page_shift, base + lane);
            u = units_of(A, q).total;
        }
        x = A.B.b > 1 ? prefix_sum(u) : u;
    };
    const int last = A.B.b > 1 ? 63 : 0;
    for (int base = 0; base < A.B.b; base += 64) {
        load(base);
        total += __builtin_amdgcn_readlane(x, last);
    }
    R = ranges(A, total);
    Start s;
    s.u = min(R.begin(group), total);
    s.u_end = min(R.begin(group + 1), total);
    s.req = s.first = 0;
    int l = 0;
    if (A.B.b > 1 && s.u < s.u_end) {
        int sum = 0;
        for (int base = 0;; base += 64) {                           // ends: the unit is one of total
            if (A.B.b > 64) load(base);                             // else x, u and q are those of the only 64
            const uint64_t past = __ballot(sum + x > s.u);
            if (past || base + 64 >= A.B.b) {
                l = past ? __ffsll((unsigned long long)past) - 1 : 0;
                s.req = base + l;
                s.first = sum + __builtin_amdgcn_readlane(x - u, l);
                break;
            }
            sum += __builtin_amdgcn_readlane(x, 63);
        }
    }
    s.q.row0 = __builtin_amdgcn_readlane(q.row0, l);
    s.q.rows = __builtin_amdgcn_readlane(q.rows, l);
    s.q.len = __builtin_amdgcn_readlane(q.len, l);
    s.q.ok = __builtin_amdgcn_readlane(q.ok, l);
    return s;
}

// Device-scope accesses to partial sums: they reach the other workgroups (on
// other XCDs too) without a cache flush.  A lane's 16 bytes go as two 64-bit
// accesses, laid out [half][lane].
__device__ __forceinline__ void put4(float *tile, int lane, f32x4 v) {
    unsigned long long *q = (unsigned long long *)tile;
    __hip_atomic_store(q + lane, __builtin_bit_cast(unsigned long long, f32x2{v[0], v[1]}), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(q + 64 + lane, __builtin_bit_cast(unsigned long long, f32x2{v[2], v[3]}), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x4 get4(const float *tile, int lane) {
    const unsigned long long *q = (const unsigned long long *)tile;
    const f32x2 a = __builtin_bit_cast(f32x2, __hip_atomic_load(q + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    const f32x2 b = __builtin_bit_cast(f32x2, __hip_atomic_load(q + 64 + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    return f32x4{a[0], a[1], b[0], b[1]};
}
__device__ __forceinline__ void put2(float *p, float a, float b) {
    __hip_atomic_store((unsigned long long *)p, __builtin_bit_cast(unsigned long long, f32x2{a, b}), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void get2(const float *p, float &a, float &b) {
    const f32x2 x = __builtin_bit_cast(f32x2, __hip_atomic_load((const unsigned long long *)p, __ATOMIC_RELAXED,
                                                                __HIP_MEMORY_SCOPE_AGENT));
    a = x[0];
    b = x[1];
}
__device__ __forceinline__ void wait_stores() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Four neighbouring dimensions of a row, rounded to nearest even.
__device__ __forceinline__ void store_out(uint16_t *dst, f32x4 x) {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    *(u32x2 *)dst = __builtin_bit_cast(u32x2, __builtin_convertvector(x, bf16x4));
}

// A group's part of a segment: the one it starts, or the one it did not.
template <int D, int RT>
__device__ __forceinline__ float *piece(const AttnArgs &A, int group, int rb, bool starts) {
    return A.part + (((int64_t)group * A.blocks + rb) * 2 + starts) * attn_piece(D, RT);
}

// RT row tiles of 16 per wave.
//
// The code on a call's path is kept short: with few steps per wave, as for a
// single token, instructions run about once each and have to be fetched.  So
// what runs once per segment is rolled up in loops.
template <int D, int BITS, int RT>
__global__ __launch_bounds__(TPB, WAVES / 4)
void tree_attn_kernel(const AttnArgs A, const int32_t *__restrict__ page_table) {
    constexpr int W = BITS == 16 ? 8 : 16;          // elements per 16-byte piece
    constexpr int KB = D / (4 * W);                 // k pieces of 16 positions
    constexpr int QB = D / 32;                      // q operands of a row tile
    constexpr int VB = D / 16;                      // v pieces of a step, output tiles of a row tile
    constexpr int NT = (RT * VB + WAVES - 1) / WAVES;               // output tiles that a wave joins
    constexpr int BR = RT * 16;
    constexpr bool AHEAD = D * BITS < 256 * 16;     // else k and v of a step do not fit the registers together
    __shared__ float2 s_ml[WAVES][RT][16];
    __shared__ uint32_t s_odd[WAVES];
    __shared__ f32x4 s_o[WAVES][RT * VB * 64];

    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    // neighbours in `at` share an XCD (workgroups go to the eight in turn)
    const int each = gridDim.x / 8, more = gridDim.x % 8, xcd = blockIdx.x % 8;
    const int at = xcd * each + min(xcd, more) + blockIdx.x / 8;
    const int group = A.blocks == 1 ? at : at / A.blocks, rb = A.blocks == 1 ? 0 : at - group * A.blocks;
    Ranges R;
    Start st = find_start(A, group, R);
    int u = __builtin_amdgcn_readfirstlane(st.u), req = __builtin_amdgcn_readfirstlane(st.req),
        rfirst = __builtin_amdgcn_readfirstlane(st.first);
    const int u_end = __builtin_amdgcn_readfirstlane(st.u_end);
    kv::Req q = st.q;
    Units un = units_of(A, q);
    const int page_mask = (1 << A.c.page_shift) - 1;
    const float c = A.scale, per_rep = 1.f / A.rep;
    const int row_base = rb * BR;                   // first of the rows (node * rep + q head)

    while (u < u_end) {
        if (u - rfirst >= un.total) {               // the next request, also past those without rows
            rfirst += un.total;
            q = kv::request(A.B, A.c.page_shift, ++req);
            q.row0 = __builtin_amdgcn_readfirstlane(q.row0);
            q.rows = __builtin_amdgcn_readfirstlane(q.rows);
            q.len = __builtin_amdgcn_readfirstlane(q.len);
            q.ok = __builtin_amdgcn_readfirstlane(q.ok);
            un = units_of(A, q);
            continue;
        }
        const int head = (u - rfirst) / un.per_seg, v0 = u - rfirst - head * un.per_seg;
        const int n = min(un.per_seg - v0, u_end - u);
        const int tokens = q.ok ? q.len + q.rows : 0;
        const int rows = q.rows * A.rep;
        if (row_base >= rows) {                     // a request of fewer row blocks
            u += n;
            continue;
        }

        // Outputs and sum of each row, in units of 2^m: m is the row's reference,
        // the maximum (log2) of probability times v scale over the first positions that
        // it sees.  Later ones may pass it by 2^11 (8 bits) or 2^32 before anything has to
        // be scaled down; then the wave starts its positions over with the higher
        // reference.  So the loop neither takes maxima nor rescales, and time depends on
        // the scores: over 8 bits 17 rows of 40 heads at 32768 positions (caches in
        // memory) take 45 us with scores of standard deviation 1.5, 84 / 130 / 157 /
        // 165 with 3 / 4 / 5 / 6, a tree of 16 at 6000 positions 13.9 and 17.5 / 19.7 /
        // 19.8 / 20.0; at worst, with scores that rise from step to step, every step has
        // those before it taken again.  Over bf16 nothing changes up to 6 (28.8 us for
        // 4 requests of 6 rows, 248 for 32 trees of 8).
        f32x4 o[RT][VB];
        float m[RT], l[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) m[rt] = NEG_INF;

        // A step takes 32 positions from t.  Pages that are none of the cache's
        // make every row that sees them NaN; page 0 is read in their place.
        // Page numbers are loaded a step ahead of the k that needs them, k a
        // step ahead of its use (AHEAD), v at the step's start (k and v both a step
        // ahead measured the same).
        const int32_t *const table = page_table + (int64_t)req * A.B.max_pages;
        u32x4 kf[2][KB];
        f32x4 ksc[2];
        int64_t chunk = 0;
        bool bad = false;
        const auto find_page = [&](int32_t page) {
            bad = page < 0 || page >= A.c.pages;
            chunk = ((int64_t)(bad ? 0 : page) * A.c.heads + head) << A.c.page_shift;
        };
        const auto load_k = [&](int t) {
            const int at = t & page_mask;
            const unsigned char *src = (const unsigned char *)A.c.k + (chunk + at) * (D * BITS / 8);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) kf[i][kb] = *(const u32x4 *)(src + (i * KB + kb) * 1024 + (uint32_t)lane * 16);
                if constexpr (BITS == 8) ksc[i] = *(const f32x4 *)(A.c.ks + chunk + at + i * 16 + (uint32_t)g * 4);
            }
        };

        const auto load_v = [&](int t, u32x4 (&vf)[VB], f32x4 (&vsc)[2]) {
            const int at = t & page_mask;
            // an 8-bit piece holds 64 positions: its first or second half
            const unsigned char *src = (const unsigned char *)A.c.v + (chunk + (at & -(4 * W))) * (D * BITS / 8) +
                                       (BITS == 8 ? (at & 32) / 4 : 0);
#pragma unroll
            for (int vb = 0; vb < VB; ++vb) {
                if constexpr (BITS == 16) {
                    vf[vb] = *(const u32x4 *)(src + vb * 1024 + (uint32_t)lane * 16);
                } else {
                    const u32x2 x = *(const u32x2 *)(src + vb * 1024 + (uint32_t)lane * 16);
                    vf[vb][0] = x[0];
                    vf[vb][1] = x[1];
                }
            }
            if constexpr (BITS == 8) {
#pragma unroll
                for (int i = 0; i < 2; ++i) vsc[i] = *(const f32x4 *)(A.c.vs + chunk + at + i * 16 + (uint32_t)g * 4);
            }
        };
        const int t_first = v0 * kUnit + w * kStep, t_end = min((v0 + n) * kUnit, tokens);
        const int32_t page_first = t_first < t_end ? table[t_first >> A.c.page_shift] : 0;

        // q operands and masks of the wave's rows; those past the last repeat it and are not written
        bf16x8 qf[RT][QB];
        uint64_t see[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int rr = min(row_base + rt * 16 + col, rows - 1), node = (int)((rr + 0.5f) * per_rep);
            const uint16_t *p = A.q + (int64_t)(q.row0 + node) * A.ldq + (head * A.rep + rr - node * A.rep) * D +
                                g * (BITS == 16 ? 8 : 16);
#pragma unroll
            for (int kb = 0; kb < QB; ++kb)
                qf[rt][kb] = as_bf16x8(*(const u32x4 *)(p + (BITS == 16 ? kb * 32 : kb / 2 * 64 + kb % 2 * 8)));
            see[rt] = (A.mask != nullptr ? A.mask[q.row0 + node] : (2ull << node) - 1) & ((2ull << (q.rows - 1)) - 1);
        }

        bool over, odd_v = false;
        do {
            over = false;
            bool fresh = true;                                      // some row may lack a reference
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                l[rt] = 0.f;
#pragma unroll
                for (int vb = 0; vb < VB; ++vb) o[rt][vb] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            int32_t page_next = 0;
            if (t_first < t_end) {
                find_page(page_first);
                if constexpr (AHEAD) load_k(t_first);
                page_next = table[min(t_first + kUnit, t_end - 1) >> A.c.page_shift];
            }
            for (int t = t_first; t < t_end; t += kUnit) {
                const bool step_bad = bad, tail = t + kStep > q.len;
                u32x4 vf[VB];
                f32x4 vsc[2];
                if constexpr (!AHEAD) load_k(t);
                else load_v(t, vf, vsc);

                // scores
                f32x4 s[RT][2];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        const u32x4 k4 = kf[i][kb];
                        if constexpr (BITS == 16) {
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt) s[rt][i] = dec::mfma(as_bf16x8(k4), qf[rt][kb], s[rt][i]);
                        } else {
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const bf16x8 a = codes_bf16(k4[2 * j], k4[2 * j + 1]);
#pragma unroll
                                for (int rt = 0; rt < RT; ++rt) s[rt][i] = dec::mfma(a, qf[rt][2 * kb + j], s[rt][i]);
                            }
                        }
                    }
                // to log2: scale times k's scale, or with masks scale alone
                f32x4 kc[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) kc[i] = BITS == 8 ? ksc[i] * c : f32x4{c, c, c, c};
                if constexpr (!AHEAD) load_v(t, vf, vsc);
                if (t + kUnit < t_end) {
                    find_page(page_next);
                    if constexpr (AHEAD) load_k(t + kUnit);
                    page_next = table[min(t + 2 * kUnit, t_end - 1) >> A.c.page_shift];
                }

                if (__builtin_expect(tail || step_bad, 0)) {
                    const int n0 = t - q.len;                       // node of the step's first position
                    if constexpr (BITS == 8) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt) s[rt][i] *= kc[i];
                            kc[i] = f32x4{1.f, 1.f, 1.f, 1.f};
                        }
                    }
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        // masked scores are -inf whatever k held
                        const uint32_t vis = n0 <= -32 ? ~0u :
                                             n0 <= 0 ? (uint32_t)((see[rt] << -n0) | ((1ull << -n0) - 1)) :
                                             n0 < 64 ? (uint32_t)(see[rt] >> n0) : 0u;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float x = step_bad ? __uint_as_float(0x7fc00000u) : s[rt][i / 4][i % 4];
                            s[rt][i / 4][i % 4] = vis >> (g * 4) & (1u << (i / 4 * 16 + i % 4)) ? x : NEG_INF;
                        }
                    }
                    if constexpr (BITS == 16) {
                        // v past the last position is 0.  A row's masked positions must
                        // not reach it as 0 * NaN: v that is not finite leaves the
                        // product and is added when the waves' results are joined.
                        bool odd = false;
                        const int left = q.rows - n0 - g * 4;
#pragma unroll
                        for (int vb = 0; vb < VB; ++vb)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int at = e / 2 * 16 + e % 2 * 2;
                                uint32_t x = at < left ? at + 1 < left ? vf[vb][e] : vf[vb][e] & 0xffffu : 0u;
                                const uint32_t keep = ((x & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) |
                                                      ((x & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u);
                                odd |= keep != ~0u;
                                vf[vb][e] = x & keep;
                            }
                        odd_v |= __any(odd);
                    } else {
                        // no scales past the last position
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (n0 + i / 4 * 16 + g * 4 + i % 4 >= q.rows) vsc[i / 4][i % 4] = 0.f;
                    }
                }
                const auto reference = [&](int rt) {                // of this step alone
                    float mx = NEG_INF;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float z = s[rt][i / 4][i % 4] * kc[i / 4][i % 4];
                        // a scale of 0 or NaN still has its sum in range
                        if constexpr (BITS == 8) z += fmaxf(__builtin_amdgcn_logf(vsc[i / 4][i % 4]), -50.f) - kBase8;
                        mx = fmaxf(mx, z);
                    }
                    return row_max(mx);
                };
                if (__builtin_expect(fresh, 0)) {
                    bool none = false;
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        if (m[rt] == NEG_INF) m[rt] = reference(rt);
                        none |= m[rt] == NEG_INF;
                    }
                    fresh = __any(none);
                }

                // scores become probabilities
                u32x4 ph[RT], pl[RT];
                bool rises[RT];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const float mc = zero_if_none(m[rt]);
                    float p[8], sum = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][i / 4][i % 4], kc[i / 4][i % 4], -mc));
                        sum += p[i];
                        if constexpr (BITS == 8) p[i] *= vsc[i / 4][i % 4];
                    }
                    if constexpr (BITS == 8) {
                        if (__builtin_expect(tail, 0)) {            // 0 times a scale that is NaN, out of the row's sight
                            asm volatile("");
#pragma unroll
                            for (int i = 0; i < 8; ++i) p[i] = s[rt][i / 4][i % 4] == NEG_INF ? 0.f : p[i];
                        }
                    }
                    rises[rt] = sum > kMostSum<BITS>;
                    if constexpr (BITS == 8)
                        rises[rt] |= max3(max3(p[0], p[1], p[2]), max3(p[3], p[4], p[5]), fmaxf(p[6], p[7])) > kMostF16;
                    l[rt] += sum;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a = p[2 * i], b = p[2 * i + 1];
                        if constexpr (BITS == 8) {
                            ph[rt][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), f16x2));
                        } else {
                            ph[rt][i] = dec::pack_hi16(a, b);
                            pl[rt][i] = dec::pack_hi16(a - __uint_as_float(__float_as_uint(a) & 0xffff0000u),
                                                       b - __uint_as_float(__float_as_uint(b) & 0xffff0000u));
                        }
                    }
                }
                bool any = false;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) any |= rises[rt];
                if (__builtin_expect(__any(any), 0)) {
                    // The rows concerned alone: the others' results stay the same to
                    // the bit.  A reference that this step has raised already does not
                    // rise again (one so large that log2 of a scale is lost in it still
                    // lets the limit be passed), so every step restarts at most once per row.
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        uint64_t of = __ballot(rises[rt]);
                        of |= of >> 32;
                        of |= of >> 16;
                        const float up = reference(rt);
                        const bool higher = (of >> col & 1) && up > m[rt];
                        m[rt] = higher ? up : m[rt];
                        over |= __any(higher) != 0;
                    }
                    if (over) break;
                }
#pragma unroll
                for (int vb = 0; vb < VB; ++vb) {
                    if constexpr (BITS == 16) {
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) {
                            o[rt][vb] = dec::mfma(as_bf16x8(vf[vb]), as_bf16x8(ph[rt]), o[rt][vb]);
                            o[rt][vb] = dec::mfma(as_bf16x8(vf[vb]), as_bf16x8(pl[rt]), o[rt][vb]);
                        }
                    } else {
                        const f16x8 a = codes_f16(vf[vb][0], vf[vb][1]);
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
                            o[rt][vb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, __builtin_bit_cast(f16x8, ph[rt]), o[rt][vb], 0, 0, 0);
                    }
                }
            }
        } while (over);

        // ---- The waves' results become one: through LDS each takes every eighth
        // output tile, of all waves.
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            l[rt] = row_sum(l[rt]);
            if (g == 0) s_ml[w][rt][col] = float2{m[rt], l[rt]};
#pragma unroll
            for (int vb = 0; vb < VB; ++vb) s_o[w][(rt * VB + vb) * 64 + lane] = o[rt][vb];
        }
        if (BITS == 16 && lane == 0) s_odd[w] = odd_v;
        __syncthreads();
        const bool whole = n == un.per_seg;
        bool odd_own = false;                                       // some of the call's own v, of any wave
        if constexpr (BITS == 16) {
#pragma unroll
            for (int k = 0; k < WAVES; ++k) odd_own |= s_odd[k] != 0;
        }
        const auto finish = [&](f32x4 z, float sum, int tile) {
            const int rr = row_base + tile / VB * 16 + col, node = (int)((rr + 0.5f) * per_rep);
            // a row that sees nothing is 0; one whose length is a fault is NaN
            const float inv = !q.ok ? __uint_as_float(0x7fc00000u) : sum == 0.f ? 0.f : 1.f / sum;
            uint16_t *dst = A.out + (int64_t)(q.row0 + node) * A.ldo + (head * A.rep + rr - node * A.rep) * D;
            if (rr < rows) store_out(dst + tile % VB * 16 + g * 4, z * inv);
        };
        // v that are not finite and that a row sees are added alone, without
        // weights: in the product they would be lost where the low half of a
        // probability, or all of it, is 0, and reach rows that do not see them.
        [[maybe_unused]] const auto not_finite = [&](f32x4 &z, float sum, int tile) {
            const int rr = min(row_base + tile / VB * 16 + col, rows - 1), node = (int)((rr + 0.5f) * per_rep);
            const uint64_t sees = (A.mask != nullptr ? A.mask[q.row0 + node] : (2ull << node) - 1) & ((2ull << (q.rows - 1)) - 1);
            const auto odd = [](float x) { return fabsf(x) < __builtin_inff() ? 0.f : x; };
            float all = 0.f;                                        // cached: dimension `col`, a fourth of the positions
            f32x4 own = {0.f, 0.f, 0.f, 0.f};                       // among the rows: as z, what the lane's row sees
            const int end = min((v0 + n) * kUnit, tokens);
#pragma unroll 1
            for (int t = v0 * kUnit; t < end; t += kStep) {
                const int64_t page = table[t >> A.c.page_shift];
                if (page < 0 || page >= A.c.pages) continue;        // rows that see it are NaN
                const uint16_t *vp = (const uint16_t *)A.c.v + (((page * A.c.heads + head) * D) << A.c.page_shift);
                const u32x4 x = *(const u32x4 *)(vp + (t & page_mask) * D + (tile % VB * 64 + lane) * W);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int at = t + e / 4 * 16 + g * 4 + e % 4;
                    if (at < q.len) all += odd(kv::bf16_f32(x[e / 2] >> (e % 2 * 16) & 0xffffu));
                }
#pragma unroll 1
                for (int at = max(t, q.len); at < min(t + kStep, end); ++at)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (sees >> (at - q.len) & 1)
                            own[i] += odd(kv::bf16_f32(vp[kv::v_elem<D, W>(at & page_mask, tile % VB * 16 + g * 4 + i)]));
            }
            all = row_sum(all);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = __shfl(all, g * 4 + i) + own[i];
                if (sum == sum && x != 0.f) z[i] = x;
            }
        };
#pragma unroll 1
        for (int tile = w; tile < RT * VB; tile += WAVES) {
            float2 ml[WAVES];
            float mx = NEG_INF, sum = 0.f;
#pragma unroll
            for (int k = 0; k < WAVES; ++k) {
                ml[k] = s_ml[k][tile / VB][col];
                mx = fmaxf(mx, ml[k].x);
            }
            const float mc = zero_if_none(mx);
            f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < WAVES; ++k) {
                const float f = __builtin_amdgcn_exp2f(ml[k].x - mc);
                sum += ml[k].y * f;
                z += s_o[k][tile * 64 + lane] * f;
            }
            if constexpr (BITS == 16) {
                const float x = (z[0] + z[1]) + (z[2] + z[3]);
                if (__builtin_expect(__any((odd_own || !(x == x)) && sum == sum), 0)) not_finite(z, sum, tile);
            }
            if (whole) {
                finish(z, sum, tile);
            } else {
                // every tile with its own copy of its rows' statistics, so that
                // a wave waits for nothing but its own stores
                float *const p = piece<D, RT>(A, group, rb, v0 == 0) + tile * kTileFloats;
                put4(p, lane, z);
                if (g == 0) put2(p + 256 + col * 2, mx, sum);
            }
        }
        if (!whole && !A.join && w < RT * VB) {
            // Count in; the last to come adds the pieces of the wave's tiles, in
            // group order.  A group starts at most one shared segment.
            wait_stores();
            const int s0 = u - v0, w0 = R.owner(s0), w1 = R.owner(s0 + un.per_seg - 1);
            uint32_t *const ctr = A.counters + ((w0 * A.blocks + rb) * WAVES + w) * kAttnCounter;
            uint32_t ticket = 0;
            if (lane == 0) ticket = __hip_atomic_fetch_add(ctr, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (__builtin_amdgcn_readfirstlane(ticket) == (uint32_t)(w1 - w0)) {
                if (lane == 0) __hip_atomic_store(ctr, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                float mx[NT], sum[NT];
                f32x4 z[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    mx[j] = NEG_INF;
                    sum[j] = 0.f;
                    z[j] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
                const auto add = [&](auto most, int k0) {           // pieces k0 .., all in flight
                    constexpr int XB = most();
                    f32x4 x[XB][NT];
                    float xm[XB][NT], xl[XB][NT];
#pragma unroll
                    for (int i = 0; i < XB; ++i) {
                        const int k = min(k0 + i, w1);
                        const float *src = piece<D, RT>(A, k, rb, k == w0);
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const float *p = src + (w + j * WAVES) * kTileFloats;
                            x[i][j] = get4(p, lane);
                            get2(p + 256 + col * 2, xm[i][j], xl[i][j]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        float mn = mx[j];
#pragma unroll
                        for (int i = 0; i < XB; ++i) mn = fmaxf(mn, xm[i][j]);
                        const float mc = zero_if_none(mn), f = __builtin_amdgcn_exp2f(mx[j] - mc);
                        z[j] *= f;
                        sum[j] *= f;
                        mx[j] = mn;
#pragma unroll
                        for (int i = 0; i < XB; ++i) {
                            // a repeated last piece is left out
                            const bool real = k0 + i <= w1;
                            const float fk = __builtin_amdgcn_exp2f(xm[i][j] - mc);
                            sum[j] += real ? xl[i][j] * fk : 0.f;
#pragma unroll
                            for (int e = 0; e < 4; ++e) z[j][e] += real ? x[i][j][e] * fk : 0.f;
                        }
                    }
                };
                if (w1 - w0 < 4) {
                    add(std::integral_constant<int, 4>(), w0);
                } else {
                    constexpr int most = NT == 1 ? 16 : 12;
#pragma unroll 1
                    for (int k0 = w0; k0 <= w1; k0 += most) add(std::integral_constant<int, most>(), k0);
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) finish(z[j], sum[j], w + j * WAVES);
            }
        }
        __syncthreads();                                            // the buffers are free for the next segment
        u += n;
    }
}

// The pieces of shared segments, where they are more than the last workgroup of
// a segment adds in good time (A.join): a workgroup per 16 x 16 output tile, a
// wave for every fourth piece, in group order.  Latency: 3.5-4.0 us for 32 times
// 8 pieces of 16 rows, 4.7-5.0 for 24 times 11 pieces of 32 rows.
template <int D, int RT>
__global__ __launch_bounds__(64 * kJoinWaves) void attn_join_kernel(const AttnArgs A) {
    constexpr int VB = D / 16, XB = 8;              // pieces of a wave in flight
    __shared__ float2 s_ml[kJoinWaves][16];
    __shared__ f32x4 s_o[kJoinWaves][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, g = lane >> 4;
    const int tile = blockIdx.x, rb = blockIdx.y % A.blocks, head = blockIdx.y / A.blocks, r = blockIdx.z;
    int total = 0, first = 0;
    Units un = {};
    kv::Req q = {};
    for (int base = 0; base < A.B.b; base += 64) {
        kv::Req ql = {};
        Units ul = {};
        if (base + lane < A.B.b) {
            ql = kv::request(A.B, A.c.page_shift, base + lane);
            ul = units_of(A, ql);
        }
        const int x = A.B.b > 1 ? prefix_sum(ul.total) : ul.total;
        if (r >= base && r < base + 64) {
            const int l = r - base;
            first = total + __builtin_amdgcn_readlane(x - ul.total, l);
            un.per_seg = __builtin_amdgcn_readlane(ul.per_seg, l);
            q.row0 = __builtin_amdgcn_readlane(ql.row0, l);
            q.rows = __builtin_amdgcn_readlane(ql.rows, l);
        }
        total += __builtin_amdgcn_readlane(x, A.B.b > 1 ? 63 : 0);
    }
    const int rows = q.rows * A.rep, row_base = rb * RT * 16;
    if (row_base + tile / VB * 16 >= rows) return;
    const Ranges R = ranges(A, total);
    first += head * un.per_seg;
    const int w0 = R.owner(first), w1 = R.owner(first + un.per_seg - 1);
    if (w0 == w1) return;                                           // written by its only group
    float mx = NEG_INF, sum = 0.f;
    f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int k0 = w0 + w; k0 <= w1; k0 += XB * kJoinWaves) {
        f32x4 x[XB];
        float2 ml[XB];
#pragma unroll
        for (int i = 0; i < XB; ++i) {
            const int k = k0 + i * kJoinWaves <= w1 ? k0 + i * kJoinWaves : k0;
            const float *p = piece<D, RT>(A, k, rb, k == w0) + tile * kTileFloats;
            const f32x2 a = *(const f32x2 *)(p + lane * 2), b = *(const f32x2 *)(p + 128 + lane * 2);
            x[i] = f32x4{a[0], a[1], b[0], b[1]};
            ml[i] = *(const float2 *)(p + 256 + col * 2);
        }
        float mn = mx;
#pragma unroll
        for (int i = 0; i < XB; ++i) mn = fmaxf(mn, ml[i].x);
        const float mc = zero_if_none(mn), f = __builtin_amdgcn_exp2f(mx - mc);
        z *= f;
        sum *= f;
        mx = mn;
#pragma unroll
        for (int i = 0; i < XB; ++i) {
            const bool real = i == 0 || k0 + i * kJoinWaves <= w1;
            const float fk = __builtin_amdgcn_exp2f(ml[i].x - mc);
            sum += real ? ml[i].y * fk : 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] += real ? x[i][e] * fk : 0.f;
        }
    }
    if (g == 0) s_ml[w][col] = float2{mx, sum};
    s_o[w][lane] = z;
    __syncthreads();
    if (w != 0) return;
    float2 ml[kJoinWaves];
    mx = NEG_INF;
#pragma unroll
    for (int k = 0; k < kJoinWaves; ++k) {
        ml[k] = s_ml[k][col];
        mx = fmaxf(mx, ml[k].x);
    }
    const float mc = zero_if_none(mx);
    sum = 0.f;
    z = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kJoinWaves; ++k) {
        const float f = __builtin_amdgcn_exp2f(ml[k].x - mc);
        sum += ml[k].y * f;
        z += s_o[k][lane] * f;
    }
    const int rr = row_base + tile / VB * 16 + col, node = (int)((rr + 0.5f) * (1.f / A.rep));
    if (rr < rows)
        store_out(A.out + (int64_t)(q.row0 + node) * A.ldo + (head * A.rep + rr - node * A.rep) * D + tile % VB * 16 + g * 4,
                  z * (sum == 0.f ? 0.f : 1.f / sum));
}

template <int D, int BITS, int RT>
hipError_t launch_tiles(const AttnArgs &A, hipStream_t s) {
    hipLaunchKernelGGL((tree_attn_kernel<D, BITS, RT>), dim3(A.groups * A.blocks), dim3(TPB), 0, s, A, A.B.page_table);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !A.join) return e;
    hipLaunchKernelGGL((attn_join_kernel<D, RT>), dim3(RT * D / 16, A.c.heads * A.blocks, A.B.b), dim3(64 * kJoinWaves), 0, s, A);
    return hipGetLastError();
}
template <int D, int BITS>
hipError_t launch(const AttnArgs &A, hipStream_t s) {
    return A.tiles == 1 ? launch_tiles<D, BITS, 1>(A, s) : launch_tiles<D, BITS, attn_tiles(D)>(A, s);
}

}  // namespace

hipError_t launch_tree_attention(const AttnArgs &A, hipStream_t s) {
    if (A.c.bits == 16)
        return A.c.d == 64 ? launch<64, 16>(A, s) : A.c.d == 128 ? launch<128, 16>(A, s) : launch<256, 16>(A, s);
    return A.c.d == 64 ? launch<64, 8>(A, s) : A.c.d == 128 ? launch<128, 8>(A, s) : launch<256, 8>(A, s);
}

}  // namespace dspk
