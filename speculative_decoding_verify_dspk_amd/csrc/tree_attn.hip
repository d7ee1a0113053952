// Attention of a round's rows over the paged cache: one token, a chain or a
// tree of up to 64 drafts per request, any number of requests, q heads in
// groups over the k/v heads.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i.k_j - max_j),
//
// j over the positions row i sees.  A (request, kv head, row block) is a
// segment; its cache positions are cut into units, and a persistent grid
// takes equal contiguous ranges of all segments' units, so ragged batches load
// every CU alike.  A segment shared by workgroups leaves partial sums in the
// workspace, which attn_join_kernel adds in workgroup order (deterministic).
//
// Within a workgroup each wave takes its own positions, so k and v go from
// memory to the matrix cores without LDS or barriers: the cache is stored in
// operand order (kv_layout.h).  Scores are computed as S^T = K Q^T, whose
// result layout (lane: one row, four neighbouring positions) is already the
// operand layout of O^T = V^T P^T; every statistic of a row lies in its
// lanes, one value each.  The waves' results are joined through LDS when a
// segment ends.
//
// Rounding: scores, maxima, sums and outputs are fp32.  A probability goes
// into the second product as the sum of two bf16 (16 significant bits): with
// one bf16 the output's error would be 1.4 times that of the final rounding
// alone, and the matrix cores have the time.  8-bit codes are exact in bf16;
// their scales multiply scores and probabilities in fp32.
#include <hip/hip_runtime.h>

#include "decode.h"
#include "kv_layout.h"

namespace dspk {
namespace {

using dec::as_bf16x8;
using dec::bf16x8;
using kv::f32x4;
using kv::u32x4;

constexpr int kWaves = 4, TPB = 64 * kWaves;
#define NEG_INF (-__builtin_inff())

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

// max and sum over the four lanes of a row (lane % 16 is the row)
__device__ __forceinline__ float row_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float row_sum(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

__device__ __forceinline__ int wave_sum(int x) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o);
    return x;
}

// Units of a request: per segment and in all.  A request with rows has at
// least one unit per segment, so that its rows are written even if nothing is
// cached or its length is a fault.
struct Units {
    int per_seg, blocks, total;
};
__device__ __forceinline__ Units units_of(const AttnArgs &A, const kv::Req &q, int unit, int block_rows) {
    Units u;
    const int tokens = q.ok ? q.len + q.rows : 0;
    u.per_seg = max(1, (tokens + unit - 1) / unit);
    u.blocks = (q.rows * A.rep + block_rows - 1) / block_rows;
    u.total = u.per_seg * u.blocks * A.c.heads;
    return u;
}

// Range of a workgroup: the first rem workgroups take q + 1 units, the others
// q.  The inverse gives the workgroup of a unit.
struct Ranges {
    int q, rem;
    __device__ __forceinline__ int begin(int w) const { return w * q + min(w, rem); }
    __device__ __forceinline__ int owner(int u) const {
        const int cut = rem * (q + 1);
        return u < cut ? u / (q + 1) : rem + (u - cut) / q;
    }
};
// All units of the call; where > = 0 also the request that holds unit `where`
// and that request's first unit.  The same on every lane; waves do it alone.
__device__ __forceinline__ int scan_units(const AttnArgs &A, int unit, int block_rows, int where, int &req, int &first) {
    const int lane = threadIdx.x & 63;
    int sum = 0;
    req = A.B.b;
    for (int base = 0; base < A.B.b; base += 64) {
        int u = 0;
        if (base + lane < A.B.b) u = units_of(A, kv::request(A.B, A.c.page_shift, base + lane), unit, block_rows).total;
        if (where >= 0 && req == A.B.b) {
            int x = u;                                              // inclusive prefix sum
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int y = __shfl_up(x, o);
                if (lane >= o) x += y;
            }
            const uint64_t past = __ballot(sum + x > where);
            if (past) {
                const int l = __ffsll((unsigned long long)past) - 1;
                req = base + l;
                first = sum + __shfl(x - u, l);
                return -1;
            }
        }
        sum += wave_sum(u);
    }
    return sum;
}

template <int D, int RT>
constexpr int slot_floats() { return RT * D * 16; }                 // a wave's partial outputs

template <int D, int BITS, int RT, int RG>
__global__ __launch_bounds__(TPB, attn_occ(D, RT))
void tree_attn_kernel(const AttnArgs A, const int32_t *__restrict__ page_table) {
    constexpr int W = BITS == 16 ? 8 : 16;          // elements per 16-byte piece
    constexpr int TS = 4 * W, TB = TS / 16;         // positions per wave step, in 16-position tiles
    constexpr int KB = D / (4 * W);                 // k pieces of a tile
    constexpr int QB = D / 32;                      // q operands of a row tile
    constexpr int VB = D / 16;                      // v pieces of a step, and output tiles of a row tile
    constexpr int PB = TS / 32;                     // probability operands of a step
    constexpr int TG = kWaves / RG, UNIT = TS * TG, BR = RG * RT * 16;
    __shared__ float s_ml[kWaves][RT][2][16];
    __shared__ f32x4 s_o[TG > 1 ? kWaves : 1][TG > 1 ? RT * VB * 64 : 1];

    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int rg = w % RG, tg = w / RG, col = lane & 15, g = lane >> 4;
    int req, rfirst;
    const int total = scan_units(A, UNIT, BR, -1, req, rfirst);
    const Ranges R{total / A.grid, total % A.grid};
    int u = __builtin_amdgcn_readfirstlane(R.begin(blockIdx.x));
    const int u_end = __builtin_amdgcn_readfirstlane(R.begin(blockIdx.x + 1));
    if (u >= u_end) return;
    scan_units(A, UNIT, BR, u, req, rfirst);
    req = __builtin_amdgcn_readfirstlane(req);
    rfirst = __builtin_amdgcn_readfirstlane(rfirst);
    const int page_mask = (1 << A.c.page_shift) - 1;
    const float c = A.scale;

    while (u < u_end) {
        kv::Req q = kv::request(A.B, A.c.page_shift, req);
        q.row0 = __builtin_amdgcn_readfirstlane(q.row0);
        q.rows = __builtin_amdgcn_readfirstlane(q.rows);
        q.len = __builtin_amdgcn_readfirstlane(q.len);
        q.ok = __builtin_amdgcn_readfirstlane(q.ok);
        const Units un = units_of(A, q, UNIT, BR);
        if (u - rfirst >= un.total) {               // also past requests without rows
            rfirst += un.total;
            ++req;
            continue;
        }
        const int seg = (u - rfirst) / un.per_seg, v0 = u - rfirst - seg * un.per_seg;
        const int n = min(un.per_seg - v0, u_end - u);
        const int rb = seg % un.blocks, head = seg / un.blocks;
        const int tokens = q.ok ? q.len + q.rows : 0;
        const int row_base = rb * BR + rg * RT * 16;                // first of the wave's rows (node * rep + q head)

        // q operands and masks of the wave's rows
        bf16x8 qf[RT][QB];
        uint64_t see[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int rr = row_base + rt * 16 + col, node = rr / A.rep;
            const bool in = node < q.rows;
            const uint16_t *p = A.q + (int64_t)(q.row0 + node) * A.ldq + (head * A.rep + rr - node * A.rep) * D;
#pragma unroll
            for (int kb = 0; kb < QB; ++kb) {
                const int d = BITS == 16 ? kb * 32 + g * 8 : kb / 2 * 64 + g * 16 + kb % 2 * 8;
                const u32x4 zero = {0u, 0u, 0u, 0u};
                qf[rt][kb] = as_bf16x8(in ? *(const u32x4 *)(p + d) : zero);
            }
            see[rt] = !in ? 0 : A.mask != nullptr ? A.mask[q.row0 + node] : (2ull << node) - 1;
        }

        f32x4 o[RT][VB];
        float m[RT], l[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            m[rt] = NEG_INF;
            l[rt] = 0.f;
#pragma unroll
            for (int vb = 0; vb < VB; ++vb) o[rt][vb] = f32x4{0.f, 0.f, 0.f, 0.f};
        }

        // One step: TS positions from t.  Pages that are none of the cache's
        // make every row that sees them NaN; page 0 is read in their place.
        // Page numbers are loaded a step ahead of the k that needs them.
        const int32_t *const table = page_table + (int64_t)req * A.B.max_pages;
        u32x4 kf[TB][KB];
        f32x4 ksc[TB];
        int64_t chunk = 0;
        bool bad = false;
        const auto load_k = [&](int t, int32_t page) {
            bad = page < 0 || page >= A.c.pages;
            chunk = (int64_t)(bad ? 0 : page) * A.c.heads + head;
            const unsigned char *src = (const unsigned char *)A.c.k + ((chunk * D) << A.c.page_shift) * (BITS / 8) +
                                       (uint32_t)(t & page_mask) * (D * BITS / 8) + lane * 16;
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) kf[tb][kb] = *(const u32x4 *)(src + (tb * KB + kb) * 1024);
            if constexpr (BITS == 8) {
                const float *s = A.c.ks + (chunk << A.c.page_shift) + (t & page_mask) + g * 4;
#pragma unroll
                for (int tb = 0; tb < TB; ++tb) ksc[tb] = *(const f32x4 *)(s + tb * 16);
            }
        };

        int t = v0 * UNIT + tg * TS;
        const int t_end = min((v0 + n) * UNIT, tokens);
        int32_t page_next = 0;
        if (t < t_end) {
            load_k(t, table[t >> A.c.page_shift]);
            page_next = table[min(t + UNIT, t_end - 1) >> A.c.page_shift];
        }
        while (t < t_end) {
            // v of this step
            u32x4 vf[VB];
            f32x4 vsc[TB];
            {
                const unsigned char *src = (const unsigned char *)A.c.v + ((chunk * D) << A.c.page_shift) * (BITS / 8) +
                                           (uint32_t)(t & page_mask) * (D * BITS / 8) + lane * 16;
#pragma unroll
                for (int vb = 0; vb < VB; ++vb) vf[vb] = *(const u32x4 *)(src + vb * 1024);
                if constexpr (BITS == 8) {
                    const float *s = A.c.vs + (chunk << A.c.page_shift) + (t & page_mask) + g * 4;
#pragma unroll
                    for (int tb = 0; tb < TB; ++tb) vsc[tb] = *(const f32x4 *)(s + tb * 16);
                }
            }
            f32x4 s[RT][TB];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int tb = 0; tb < TB; ++tb) s[rt][tb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    if constexpr (BITS == 16) {
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
                            s[rt][tb] = dec::mfma(as_bf16x8(kf[tb][kb]), qf[rt][kb], s[rt][tb]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const bf16x8 a = codes_bf16(kf[tb][kb][2 * j], kf[tb][kb][2 * j + 1]);
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt) s[rt][tb] = dec::mfma(a, qf[rt][2 * kb + j], s[rt][tb]);
                        }
                        // one piece at a time: the scheduler would otherwise decode all of k first and spill
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            const bool step_bad = bad, tail = t + TS > q.len;
            const int64_t step_chunk = chunk;
            if constexpr (BITS == 8) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int tb = 0; tb < TB; ++tb) s[rt][tb] *= ksc[tb];
            }
            const int t_next = t + UNIT;
            if (t_next < t_end) {
                load_k(t_next, page_next);
                page_next = table[min(t_next + UNIT, t_end - 1) >> A.c.page_shift];
            }

            bool odd_v = false;
            if (tail || step_bad) {
                // masked scores are -inf whatever k held; v past the last position is 0
#pragma unroll
                for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int node = t + tb * 16 + g * 4 + i - q.len;
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) {
                            const bool vis = node < 0 || (node < q.rows && (see[rt] >> (node & 63) & 1));
                            const float x = step_bad ? __uint_as_float(0x7fc00000u) : s[rt][tb][i];
                            s[rt][tb][i] = vis ? x : NEG_INF;
                        }
                    }
                if constexpr (BITS == 16) {
                    // A row's masked positions must not reach it as 0 * NaN:
                    // v that is not finite leaves the product and is added
                    // to the rows that see it.
                    bool odd = false;
#pragma unroll
                    for (int vb = 0; vb < VB; ++vb)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int node = t + e / 2 * 16 + g * 4 + e % 2 * 2 - q.len;
                            uint32_t x = vf[vb][e];
                            if (node >= q.rows) x &= 0xffff0000u;
                            if (node + 1 >= q.rows) x &= 0xffffu;
                            const bool lo = (x & 0x7f80u) == 0x7f80u, hi = (x & 0x7f800000u) == 0x7f800000u;
                            odd |= lo || hi;
                            if (lo) x &= 0xffff0000u;
                            if (hi) x &= 0xffffu;
                            vf[vb][e] = x;
                        }
                    odd_v = __any(odd);
                }
            }

            // running maximum and sum; scores become probabilities
            bf16x8 ph[RT][PB], pl[RT][PB];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                float mx = m[rt];
#pragma unroll
                for (int tb = 0; tb < TB; ++tb)
                    mx = fmaxf(fmaxf(fmaxf(mx, s[rt][tb][0]), fmaxf(s[rt][tb][1], s[rt][tb][2])), s[rt][tb][3]);
                mx = row_max(mx);
                const float mc = mx == NEG_INF ? 0.f : mx * c;      // nothing seen yet: exp2(-inf) = 0 below
                if (__any(mx > m[rt])) {
                    const float f = __builtin_amdgcn_exp2f(m[rt] * c - mc);
                    l[rt] *= f;
#pragma unroll
                    for (int vb = 0; vb < VB; ++vb) o[rt][vb] *= f;
                    m[rt] = mx;
                }
                float sum = 0.f;
                uint32_t hw[TB * 2], lw[TB * 2];
#pragma unroll
                for (int tb = 0; tb < TB; ++tb) {
                    float p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][tb][i], c, -mc));
                        sum += p[i];
                        if constexpr (BITS == 8) {
                            const float x = p[i] * vsc[tb][i];
                            p[i] = tail && s[rt][tb][i] == NEG_INF ? 0.f : x;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float a = p[2 * i], b = p[2 * i + 1];
                        hw[tb * 2 + i] = dec::pack_hi16(a, b);
                        lw[tb * 2 + i] = dec::pack_hi16(a - __uint_as_float(__float_as_uint(a) & 0xffff0000u),
                                                        b - __uint_as_float(__float_as_uint(b) & 0xffff0000u));
                    }
                }
                l[rt] += sum;
#pragma unroll
                for (int j = 0; j < PB; ++j) {
                    ph[rt][j] = as_bf16x8(u32x4{hw[4 * j], hw[4 * j + 1], hw[4 * j + 2], hw[4 * j + 3]});
                    pl[rt][j] = as_bf16x8(u32x4{lw[4 * j], lw[4 * j + 1], lw[4 * j + 2], lw[4 * j + 3]});
                }
            }
            if constexpr (BITS == 16) {
                if (odd_v) {
                    const uint16_t *vp = (const uint16_t *)A.c.v + ((step_chunk * D) << A.c.page_shift);
                    const int last = min(TS, tokens - t);
                    for (int tt = 0; tt < last; ++tt) {
                        const int node = t + tt - q.len;
#pragma unroll
                        for (int vb = 0; vb < VB; ++vb)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float x = kv::bf16_f32(
                                    vp[kv::v_elem<D, W>((t & page_mask) + tt, vb * 16 + g * 4 + i)]);
                                if (!(fabsf(x) < __builtin_inff())) {
#pragma unroll
                                    for (int rt = 0; rt < RT; ++rt)
                                        if (node < 0 || (see[rt] >> (node & 63) & 1)) o[rt][vb][i] += x;
                                }
                            }
                    }
                }
            }
#pragma unroll
            for (int vb = 0; vb < VB; ++vb)
#pragma unroll
                for (int j = 0; j < PB; ++j) {
                    const bf16x8 a = BITS == 16 ? as_bf16x8(vf[vb]) : codes_bf16(vf[vb][2 * j], vf[vb][2 * j + 1]);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        o[rt][vb] = dec::mfma(a, ph[rt][j], o[rt][vb]);
                        o[rt][vb] = dec::mfma(a, pl[rt][j], o[rt][vb]);
                    }
                    if constexpr (BITS == 8) __builtin_amdgcn_sched_barrier(0);
                }
            t = t_next;
        }

        // ---- the token groups' results become one
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) l[rt] = row_sum(l[rt]);
        if constexpr (TG > 1) {
            if (g == 0) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    s_ml[w][rt][0][col] = m[rt];
                    s_ml[w][rt][1][col] = l[rt];
                }
            }
            __syncthreads();
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                float mx = NEG_INF, sum = 0.f;
#pragma unroll
                for (int k = 0; k < TG; ++k) mx = fmaxf(mx, s_ml[k * RG + rg][rt][0][col]);
                const float mc = mx == NEG_INF ? 0.f : mx * c;
#pragma unroll
                for (int k = 0; k < TG; ++k)
                    sum += s_ml[k * RG + rg][rt][1][col] * __builtin_amdgcn_exp2f(s_ml[k * RG + rg][rt][0][col] * c - mc);
                const float f = __builtin_amdgcn_exp2f(m[rt] * c - mc);
#pragma unroll
                for (int vb = 0; vb < VB; ++vb) s_o[w][(rt * VB + vb) * 64 + lane] = o[rt][vb] * f;
                m[rt] = mx;
                l[rt] = sum;
            }
            __syncthreads();
        }

        // ---- output rows, or partial sums: wave tg of a row group writes every TG-th tile
        const bool whole = n == un.per_seg;
        const int64_t slot = ((int64_t)blockIdx.x * 2 + (v0 == 0 ? 1 : 0)) * RG + rg;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int rr = row_base + rt * 16 + col, node = rr / A.rep;
            const bool in = node < q.rows;
            uint16_t *dst = A.out + (int64_t)(q.row0 + node) * A.ldo + (head * A.rep + rr - node * A.rep) * D;
            // a row that sees nothing is 0; one whose length is a fault is NaN
            const float inv = !q.ok ? __uint_as_float(0x7fc00000u) : l[rt] == 0.f ? 0.f : 1.f / l[rt];
#pragma unroll
            for (int vb = 0; vb < VB; ++vb) {
                if (TG > 1 && vb % TG != tg) continue;
                f32x4 x = o[rt][vb];
                if constexpr (TG > 1) {
                    x = s_o[rg][(rt * VB + vb) * 64 + lane];
#pragma unroll
                    for (int k = 1; k < TG; ++k) x += s_o[k * RG + rg][(rt * VB + vb) * 64 + lane];
                }
                if (whole) {
                    x *= inv;
                    if (in) {
                        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
                        u32x2 y;
                        y[0] = (uint32_t)dec::f2bf16(x[0]) | (uint32_t)dec::f2bf16(x[1]) << 16;
                        y[1] = (uint32_t)dec::f2bf16(x[2]) | (uint32_t)dec::f2bf16(x[3]) << 16;
                        *(u32x2 *)(dst + vb * 16 + g * 4) = y;
                    }
                } else {
                    *((f32x4 *)(A.part + slot * slot_floats<D, RT>()) + (rt * VB + vb) * 64 + lane) = x;
                }
            }
            if (!whole && tg == 0 && g == 0) {
                float *ml = A.part_ml + (slot * RT + rt) * 32;
                ml[col] = m[rt];
                ml[16 + col] = l[rt];
            }
        }
        if constexpr (TG > 1) __syncthreads();                      // the buffers are free for the next segment
        u += n;
    }
}

// Adds the partial sums of segments that several workgroups share.  A
// workgroup of this kernel takes 16 rows and 32 dimensions of one segment;
// its waves take every fourth contributor and are joined through LDS.
template <int D, int RT, int RG>
__global__ __launch_bounds__(TPB) void attn_join_kernel(const AttnArgs A, const int unit, const int blocks) {
    constexpr int VB = D / 16, BR = RG * RT * 16;
    __shared__ float s_ml[kWaves][2][16];
    __shared__ f32x4 s_o[kWaves][2][64];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    int at = blockIdx.x;
    const int vp = at % (VB / 2);
    at /= VB / 2;
    const int rt = at % RT;
    at /= RT;
    const int rg = at % RG;
    at /= RG;
    const int rb = at % blocks;
    at /= blocks;
    const int head = at % A.c.heads, r = at / A.c.heads;
    const kv::Req q = kv::request(A.B, A.c.page_shift, r);
    const Units un = units_of(A, q, unit, BR);
    if (rb >= un.blocks || rb * BR + (rg * RT + rt) * 16 >= q.rows * A.rep) return;
    int total = 0, first = 0;
    for (int base = 0; base < A.B.b; base += 64) {
        int x = 0;
        if (base + lane < A.B.b) x = units_of(A, kv::request(A.B, A.c.page_shift, base + lane), unit, BR).total;
        first += wave_sum(base + lane < r ? x : 0);
        total += wave_sum(x);
    }
    const Ranges R{total / A.grid, total % A.grid};
    first += (head * un.blocks + rb) * un.per_seg;
    const int w0 = R.owner(first), w1 = R.owner(first + un.per_seg - 1);
    if (w0 == w1) return;                                           // written by its only workgroup
    const float c = A.scale;
    float m = NEG_INF, l = 0.f;
    f32x4 o[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    for (int k = w0 + w; k <= w1; k += kWaves) {
        const int64_t slot = ((int64_t)k * 2 + (k == w0 ? 1 : 0)) * RG + rg;
        const float *ml = A.part_ml + (slot * RT + rt) * 32;
        const f32x4 *po = (const f32x4 *)(A.part + slot * slot_floats<D, RT>()) + (rt * VB + vp * 2) * 64 + lane;
        const float mk = ml[col], lk = ml[16 + col];
        const f32x4 x0 = po[0], x1 = po[64];
        const float mx = fmaxf(m, mk), mc = mx == NEG_INF ? 0.f : mx * c;
        const float f = __builtin_amdgcn_exp2f(m * c - mc), fk = __builtin_amdgcn_exp2f(mk * c - mc);
        o[0] = o[0] * f + x0 * fk;
        o[1] = o[1] * f + x1 * fk;
        l = l * f + lk * fk;
        m = mx;
    }
    if (g == 0) {
        s_ml[w][0][col] = m;
        s_ml[w][1][col] = l;
    }
    s_o[w][0][lane] = o[0];
    s_o[w][1][lane] = o[1];
    __syncthreads();
    if (w >= 2) return;
    float mx = NEG_INF;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) mx = fmaxf(mx, s_ml[k][0][col]);
    const float mc = mx == NEG_INF ? 0.f : mx * c;
    float sum = 0.f;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
        const float f = __builtin_amdgcn_exp2f(s_ml[k][0][col] * c - mc);
        sum += s_ml[k][1][col] * f;
        x += s_o[k][w][lane] * f;
    }
    const int rr = rb * BR + (rg * RT + rt) * 16 + col, node = rr / A.rep;
    if (node >= q.rows) return;
    x *= sum == 0.f ? 0.f : 1.f / sum;
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    u32x2 y;
    y[0] = (uint32_t)dec::f2bf16(x[0]) | (uint32_t)dec::f2bf16(x[1]) << 16;
    y[1] = (uint32_t)dec::f2bf16(x[2]) | (uint32_t)dec::f2bf16(x[3]) << 16;
    *(u32x2 *)(A.out + (int64_t)(q.row0 + node) * A.ldo + (head * A.rep + rr - node * A.rep) * D + (vp * 2 + w) * 16 +
               g * 4) = y;
}

template <int D, int BITS, int RT, int RG>
hipError_t launch(const AttnArgs &A, const AttnPlan &p, hipStream_t s) {
    hipLaunchKernelGGL((tree_attn_kernel<D, BITS, RT, RG>), dim3(p.grid), dim3(TPB), 0, s, A,
                       A.B.page_table);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.split) return e;
    const int grid = A.B.b * A.c.heads * p.blocks * RG * RT * (D / 32);
    hipLaunchKernelGGL((attn_join_kernel<D, RT, RG>), dim3(grid), dim3(TPB), 0, s, A, p.unit, p.blocks);
    return hipGetLastError();
}

template <int D, int BITS>
hipError_t by_rows(const AttnArgs &A, const AttnPlan &p, hipStream_t s) {
    if constexpr (D == 256) {
        if (p.rg == 4) return launch<D, BITS, 2, 4>(A, p, s);
        if (p.rg == 2) return launch<D, BITS, 2, 2>(A, p, s);
    } else {
        if (p.rg == 4) return launch<D, BITS, 4, 4>(A, p, s);
        if (p.rg == 2) return p.rt == 3 ? launch<D, BITS, 3, 2>(A, p, s) : launch<D, BITS, 4, 2>(A, p, s);
        if (p.rt == 4) return launch<D, BITS, 4, 1>(A, p, s);
    }
    return p.rt == 1 ? launch<D, BITS, 1, 1>(A, p, s) : launch<D, BITS, 2, 1>(A, p, s);
}

}  // namespace

hipError_t launch_tree_attention(const AttnArgs &A, const AttnPlan &p, hipStream_t s) {
    if (A.c.bits == 16)
        return A.c.d == 64 ? by_rows<64, 16>(A, p, s) : A.c.d == 128 ? by_rows<128, 16>(A, p, s) : by_rows<256, 16>(A, p, s);
    return A.c.d == 64 ? by_rows<64, 8>(A, p, s) : A.c.d == 128 ? by_rows<128, 8>(A, p, s) : by_rows<256, 8>(A, p, s);
}

}  // namespace dspk
