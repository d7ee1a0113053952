// Rows into the paged cache and out of it:
//   append_kernel   q/k/v rows of the projections -> RMS norm of each q and k
//                   head, rotation by position, q rows out, k/v rows into the
//                   cache (8-bit caches: codes and one scale per position and
//                   head), in one launch;
//   kv_read_kernel  cache entries -> rows;
//   kv_commit_kernel  the entries of a tree's accepted path moved together.
//
// The cache keeps k and v in the order the matrix cores take them
// (kv_layout.h), so v's positions lie next to each other: a workgroup takes
// the rows of one 64-position block of one request and head and turns v
// through LDS, so that whole 16-byte pieces are written wherever the rows
// fill them (32 positions, half an 8-bit piece, where there are few blocks).
// q's workgroups take rows and keep four loads per lane on their
// way (one: 51 us for the prompts below).
//
// Bound by memory traffic for prompts, by the latency of one load-compute-store
// chain (and by the launch) for verify rows.  Measured on MI355X, passes back to
// back: norm, rotation and store of 6250 prompt rows of 40 + 8 + 8 heads of 128
// 41 us (179 MB, 4.3 TB/s; a large copy reaches 4.8), of one row 4.3 us, of 24
// rows 4.7; 8192 rows of 8 + 8 heads into 8 bits 13 us and back 11.5 (51 MB
// each); 24 rows 4.8 and 3.3.
#include <hip/hip_runtime.h>

#include "kv_layout.h"

namespace dspk {
namespace {

using kv::u32x4;
using kv::f32x4;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int TPB = kRowThreads;
constexpr int kChunk = 16;          // k/v positions whose cosines are held at a time

// Eight lanes' worth of geometry: a head's row is held by D / 8 lanes, eight
// neighbouring dimensions each.
template <int D>
struct Geo {
    static constexpr int L = D / 8;          // lanes per row
    static constexpr int R = TPB / L;        // rows of a workgroup pass
};

// Eight neighbouring elements as they lie in memory, and as floats.
template <bool F32>
struct Raw8 {
    u32x4 v[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        const u32x4 *q = (const u32x4 *)((const char *)p + i * (F32 ? 4 : 2));
        v[0] = q[0];
        if constexpr (F32) v[1] = q[1];
    }
    __device__ __forceinline__ void clear() {
        v[0] = u32x4{0u, 0u, 0u, 0u};
        if constexpr (F32) v[1] = v[0];
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (F32) {
                x[e] = __uint_as_float(v[0][e]);
                x[e + 4] = __uint_as_float(v[1][e]);
            } else {
                x[2 * e] = __uint_as_float(v[0][e] << 16);
                x[2 * e + 1] = __uint_as_float(v[0][e] & 0xffff0000u);
            }
        }
    }
};

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x4 bf16_8(const float (&x)[8]) {         // round to nearest even
    u32x4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        r[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{x[2 * e], x[2 * e + 1]}), bf16x2));
    return r;
}

// The value of another lane, by a permutation that needs no address: CTRL of
// the data-parallel primitives, or with M lane ^ M.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
template <int M>
__device__ __forceinline__ float lane_xor(float x) {
    return __uint_as_float(__builtin_amdgcn_ds_swizzle(__float_as_uint(x), M << 10 | 0x1f));
}
// f over the L lanes of a row, L = 8, 16 or 32: within four lanes, then eight,
// sixteen (mirrored halves are equal by then) and thirty-two.
template <int L, typename F>
__device__ __forceinline__ float over_row(float x, F f) {
    x = f(x, dpp<0xb1>(x));
    x = f(x, dpp<0x4e>(x));
    x = f(x, dpp<0x141>(x));
    if constexpr (L >= 16) x = f(x, dpp<0x140>(x));
    if constexpr (L >= 32) x = f(x, lane_xor<16>(x));
    return x;
}

// 1 / sqrt(mean(x^2) + eps) of a head's row, the sum in fp32.
template <int D>
__device__ __forceinline__ float norm_factor(const float (&x)[8], float eps) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s += x[e] * x[e];
    s = over_row<Geo<D>::L>(s, [](float a, float b) { return a + b; });
    return rsqrtf(s * (1.f / D) + eps);
}

__device__ __forceinline__ int next_pow2(int x) { return x <= 1 ? 1 : 1 << (32 - __clz(x - 1)); }

// Turns per position as a fraction of 2^64, and cos and sin of a position's
// angle.  Counting turns in 64-bit fixed point keeps far positions exact: at
// position 10^6 an fp32 product would be off by 0.06 radians.
__device__ __forceinline__ uint64_t turns(float freq) {
    const double t = (double)freq * 0.15915494309189533577, part = t - floor(t);
    return part < 1.0 ? (uint64_t)(part * 0x1p64) : 0;
}
__device__ __forceinline__ void turn(int32_t position, uint64_t per, float &c, float &s) {
    const int32_t t = (int32_t)(uint32_t)(((uint64_t)(int64_t)position * per) >> 32);      // of 2^32
    sincospif((float)t * 0x1p-31f, &s, &c);
}

// What norm and rotation do to the eight dimensions of a lane, for one row:
// x -> f (x * cw + partner * sw), f the norm's factor; cosines, sines and
// weights of the lane and of its partners are folded together.
struct Turn8 {
    float cw[8], sw[8];
};
// The part that is the same for all rows: weights, and the partners' with the
// sign of their sines (0 where nothing turns); the lane's place in a table.
struct Lane8 {
    float own[8], other[8];
    int at;                     // first of the lane's frequencies
    bool in;
};
__device__ __forceinline__ void get8(const float *p, float (&x)[8]) {
    const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = a[e], x[e + 4] = b[e];
}
__device__ __forceinline__ Lane8 make_lane(int oct, int rot, int interleaved, const float *w) {
    Lane8 r;
    const int d0 = oct * 8, h = rot / 2;            // h is a multiple of 8
    r.in = d0 < rot;
    const bool first = d0 < h;
    r.at = !r.in ? 0 : interleaved ? d0 / 2 : first ? d0 : d0 - h;
#pragma unroll
    for (int e = 0; e < 8; ++e) r.own[e] = r.other[e] = 1.f;
    if (w != nullptr) {
        get8(w + d0, r.own);
        get8(w + (!r.in || interleaved ? d0 : first ? d0 + h : d0 - h), r.other);
    }
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float a = r.other[e];
            r.other[e] = -r.other[e + 1];
            r.other[e + 1] = a;
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) r.other[e] = !r.in ? 0.f : !interleaved && first ? -r.other[e] : r.other[e];
    return r;
}
// cs: the row's cosines, sn: its sines.
__device__ __forceinline__ Turn8 make_turn(const Lane8 &l, int rot, int interleaved, const float *cs, const float *sn) {
    Turn8 r;
    float c[8], s[8];
    if (rot == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r.cw[e] = l.own[e], r.sw[e] = 0.f;
        return r;
    }
    if (interleaved) {
        const f32x4 a = *(const f32x4 *)(cs + l.at), b = *(const f32x4 *)(sn + l.at);
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = a[e / 2], s[e] = b[e / 2];
    } else {
        get8(cs + l.at, c);
        get8(sn + l.at, s);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        r.cw[e] = l.in ? c[e] * l.own[e] : l.own[e];
        r.sw[e] = s[e] * l.other[e];
    }
    return r;
}
// All lanes of the wave take part.
template <int D>
__device__ __forceinline__ void norm_turn(float (&x)[8], bool norm, float eps, int rot, int interleaved, const Turn8 &t) {
    const float f = norm ? norm_factor<D>(x, eps) : 1.f;
    float p[8];
    if (rot == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = 0.f;
    } else if (interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = x[e ^ 1];
    } else if (rot == D) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (D == 128) p[e] = dpp<0x128>(x[e]);        // eight lanes on, of sixteen
            else p[e] = lane_xor<Geo<D>::L / 2>(x[e]);
        }
    } else {
        const int d0 = threadIdx.x % Geo<D>::L * 8;
        const int src = (threadIdx.x & 63) + (d0 >= rot ? 0 : d0 < rot / 2 ? rot / 16 : -(rot / 16));
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = __shfl(x[e], src);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = f * (x[e] * t.cw[e] + p[e] * t.sw[e]);
}

// A head's row as 8-bit codes: scale = max|x| / 127, code = round(x * (127 /
// max|x|)), half to even.  A row with a value that is not finite has scale NaN
// (every value reads back as NaN); one below 4e-37, whose 127 / max|x|
// would overflow, reads back as zeros.
template <int D>
__device__ __forceinline__ u32x2 codes8(const float (&x)[8], float &scale) {
    uint32_t top = 0;                              // bit patterns of magnitudes order like them, NaN on top
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
    top = __float_as_uint(over_row<Geo<D>::L>(__uint_as_float(top), [](float a, float b) {
        return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
    }));
    const float t = __uint_as_float(top), inv = 127.f / t;
    const bool held = top < 0x7f800000u && inv < __uint_as_float(0x7f800000u);
    scale = top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : held ? t / 127.f : 0.f;
    u32x2 r = {0u, 0u};
    if (held) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = (int)fminf(fmaxf(rintf(x[e] * inv), -127.f), 127.f);
            r[e / 4] |= (uint32_t)(c & 0xff) << (8 * (e % 4));
        }
    }
    return r;
}

// The rows of request q that lie in block tb of its touched blocks of 2^bs
// positions: positions base + lo .. base + hi - 1.
struct Span {
    int32_t base, lo, hi;
};
__device__ __forceinline__ Span span(const kv::Req &q, int tb, int bs = kBlockShift) {
    Span s;
    s.base = ((q.len >> bs) + tb) << bs;
    s.lo = max(q.len - s.base, 0);
    s.hi = min(q.len + q.rows - s.base, 1 << bs);
    return s;
}
// The page of a position, or -1 where its number is none of the cache's.
__device__ __forceinline__ int64_t page_of(const KvCache &c, const AttnBatch &B, int r, int32_t position) {
    const int64_t p = B.page_table[(int64_t)r * B.max_pages + (position >> c.page_shift)];
    return p >= 0 && p < c.pages ? p : -1;
}

template <int D, int BITS>
__device__ __forceinline__ int64_t chunk_elems(const KvCache &c) {
    return (int64_t)D << c.page_shift;
}

// Rows are taken in chunks whose cosines and sines are worked out first, each
// once per workgroup; the chunk's elements are on their way meanwhile.
template <int D, int BITS, bool F32>
__global__ __launch_bounds__(TPB) void append_kernel(const AppendArgs A) {
    constexpr int L = Geo<D>::L, R = Geo<D>::R, W = BITS == 16 ? 8 : 16;
    constexpr int CH = kChunk > R ? kChunk : R, NP = CH / R;        // k/v positions of a chunk, passes over them
    typedef typename std::conditional<BITS == 16, uint16_t, uint8_t>::type E;
    constexpr int VS = D + 16 / (int)sizeof(E);                     // padded row of the turned v
    __shared__ __attribute__((aligned(16))) float s_cs[2][CH * D / 2];
    __shared__ __attribute__((aligned(16))) E s_v[kBlockTokens * VS];
    const int tid = threadIdx.x, oct = tid % L, slot = tid / L, rot = A.inv_freq != nullptr ? A.rot : 0, h = rot / 2;
    const int kv_blocks = A.g.kv_blocks, nb = A.g.nb, bs = A.g.bs;

    if ((int)blockIdx.x >= kv_blocks) {
        // ---- q heads of q_rows rows of a request, or a slice of them
        const int q_rows = A.g.q_rows, q_blocks = A.g.q_blocks, slices = A.g.slices;
        const int at = blockIdx.x - kv_blocks, sl = at % slices, r = at / slices / q_blocks, i0 = at / slices % q_blocks * q_rows;
        const kv::Req q = kv::request(A.B, A.c.page_shift, r);
        const int n = min(q_rows, q.rows - i0);
        if (n <= 0) return;
        const int p2 = next_pow2(h), f = tid & (p2 - 1);            // a frequency per thread
        const int passes = (A.q_heads + R - 1) / R;                 // of a row's heads
        constexpr int AT = 4;                                       // passes whose elements are on their way
        Raw8<F32> next[AT];
        const auto load = [&](int i, int j, int p) {
            const int hd = p * R + slot;
            if (hd < A.q_heads) next[j].load(A.q, (int64_t)(q.row0 + i0 + i) * A.ldq + hd * D + oct * 8);
        };
#pragma unroll
        for (int j = 0; j < AT; ++j) {
            next[j].clear();
            load(0, j, sl + j * slices);
        }
        const Lane8 ln = make_lane(oct, rot, A.interleaved, A.qw);
        if (rot && f < h) {
            const uint64_t per = turns(A.inv_freq[f]);
            for (int i = tid / p2; i < n; i += TPB / p2) {
                const int row = i0 + i;
                turn(A.positions != nullptr ? A.positions[q.row0 + row] : q.len + row, per, s_cs[0][i * h + f], s_cs[1][i * h + f]);
            }
        }
        __syncthreads();
        for (int pb = sl; pb < passes; pb += AT * slices) {
            if (pb != sl) {
#pragma unroll
                for (int j = 0; j < AT; ++j) load(0, j, pb + j * slices);
            }
            for (int i = 0; i < n; ++i) {
                const Turn8 t = make_turn(ln, rot, A.interleaved, s_cs[0] + i * h, s_cs[1] + i * h);
#pragma unroll
                for (int j = 0; j < AT; ++j) {
                    const int p = pb + j * slices, hd = p * R + slot;
                    if (p >= passes) break;                         // the same for all
                    float x[8];
                    next[j].get(x);
                    if (i + 1 < n) load(i + 1, j, p);
                    norm_turn<D>(x, A.qw != nullptr, A.eps, rot, A.interleaved, t);
                    if (hd < A.q_heads)
                        *(u32x4 *)(A.q_out + (int64_t)(q.row0 + i0 + i) * A.ldqo + hd * D + oct * 8) = bf16_8(x);
                }
            }
        }
        return;
    }

    // ---- the k/v rows of one block of one request and head
    const int head = blockIdx.x % A.c.heads, tb = blockIdx.x / A.c.heads % nb, r = blockIdx.x / A.c.heads / nb;
    const kv::Req q = kv::request(A.B, A.c.page_shift, r);
    if (!q.ok) return;
    const Span sp = span(q, tb, bs);
    if (sp.lo >= sp.hi) return;
    const int64_t page = page_of(A.c, A.B, r, sp.base);
    const int t0 = sp.base & ((1 << A.c.page_shift) - 1);
    const int64_t chunk = page * A.c.heads + head;
    E *const kd = (E *)A.c.k + chunk * chunk_elems<D, BITS>(A.c), *const vd = (E *)A.c.v + chunk * chunk_elems<D, BITS>(A.c);
    const int row0 = q.row0 + sp.base - q.len;                      // row of the block's position 0
    const Lane8 ln = make_lane(oct, rot, A.interleaved, A.kw);
    uint64_t per_turn = 0;
    if (rot && (tid & (next_pow2(h) - 1)) < h) per_turn = turns(A.inv_freq[tid & (next_pow2(h) - 1)]);

    for (int c0 = sp.lo / CH * CH; c0 < sp.hi; c0 += CH) {
        Raw8<F32> kr[NP], vr[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int t = c0 + p * R + slot;
            if (t >= sp.lo && t < sp.hi) {
                kr[p].load(A.k, (row0 + t) * A.ldk + head * D + oct * 8);
                vr[p].load(A.v, (row0 + t) * A.ldv + head * D + oct * 8);
            } else {
                kr[p].clear();
                vr[p].clear();
            }
        }
        if (page < 0) return;                                       // asked after the loads have left; nothing is stored
        if (rot) {
            __syncthreads();                                        // the previous chunk has read its table
            const int hi = min(sp.hi, c0 + CH), p2 = next_pow2(h), f = tid & (p2 - 1);
            if (f < h) {
                for (int t = max(sp.lo, c0) + tid / p2; t < hi; t += TPB / p2)
                    turn(A.positions != nullptr ? A.positions[row0 + t] : sp.base + t, per_turn, s_cs[0][(t - c0) * h + f],
                         s_cs[1][(t - c0) * h + f]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int t = c0 + p * R + slot;
            const bool in = t >= sp.lo && t < sp.hi;
            if (c0 + p * R >= sp.hi || c0 + p * R + R <= sp.lo) continue;   // no row of the pass: the same for all
            float x[8], y[8];
            kr[p].get(x);
            vr[p].get(y);
            if (rot || A.kw != nullptr) {
                const int of = (t - c0) * h;
                norm_turn<D>(x, A.kw != nullptr, A.eps, rot, A.interleaved,
                             make_turn(ln, rot, A.interleaved, s_cs[0] + of, s_cs[1] + of));
            }
            E *const kp = kd + kv::k_piece<D, W>(t0 + t, oct * 8) + (BITS == 8 ? oct % 2 * 8 : 0);
            if constexpr (BITS == 16) {
                if (in) {
                    *(u32x4 *)kp = bf16_8(x);
                    *(u32x4 *)(s_v + t * VS + oct * 8) = bf16_8(y);
                }
            } else {
                float sk, sv;
                const u32x2 a = codes8<D>(x, sk), b = codes8<D>(y, sv);
                if (in) {
                    *(u32x2 *)kp = a;
                    *(u32x2 *)(s_v + t * VS + oct * 8) = b;
                    if (oct == 0) {
                        const int64_t si = (chunk << A.c.page_shift) + t0 + t;
                        A.c.ks[si] = sk;
                        A.c.vs[si] = sv;
                    }
                }
            }
        }
    }
    __syncthreads();
    // the turned v; a whole block of 8-bit pieces 16 bytes at a time (8192 rows
    // there and back 24.3 us, with halves 25.0)
    constexpr int per = 64 * (D / 16);                              // pieces of 4W positions
    if (BITS == 8 && sp.hi - sp.lo == kBlockTokens) {
        for (int i = tid; i < per; i += TPB) {
            const int vb = i / 64, g = i / 16 % 4, d = vb * 16 + i % 16;
            E e[W];
#pragma unroll
            for (int j = 0; j < W; ++j) e[j] = s_v[(g * 4 + j / 4 * 16 + j % 4) * VS + d];
            *(u32x4 *)(vd + kv::v_elem<D, W>(t0 + g * 4, d)) = __builtin_bit_cast(u32x4, e);
        }
        return;
    }
    // of every piece the 8 elements that lie in 32 positions (all of a bf16
    // piece, half of an 8-bit one), where they hold rows
    typedef typename std::conditional<BITS == 16, u32x4, u32x2>::type P8;
    for (int i = sp.lo / 32 * per + tid; i < (sp.hi + 31) / 32 * per; i += TPB) {
        const int sb = i / per, vb = i / 64 % (D / 16), g = i / 16 % 4, d = vb * 16 + i % 16;
        const int first = sb * 32 + g * 4;                          // their positions: first + 16 jj + i
        if (first >= sp.hi || first + 19 < sp.lo) continue;
        E *const dst = vd + kv::v_elem<D, W>(t0 + first, d);
        if (first >= sp.lo && first + 19 < sp.hi) {
            E e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = s_v[(first + j / 4 * 16 + j % 4) * VS + d];
            *(P8 *)dst = __builtin_bit_cast(P8, e);
        } else {
            for (int j = 0; j < 8; ++j) {
                const int t = first + j / 4 * 16 + j % 4;
                if (t >= sp.lo && t < sp.hi) dst[j] = s_v[t * VS + d];
            }
        }
    }
}

// Rows q.len .. of the requests, as an append with the same batch wrote them.
// Rows whose length or page is a fault read back as NaN.
template <int D, int BITS, bool F32>
__global__ __launch_bounds__(TPB) void kv_read_kernel(const ReadArgs A) {
    constexpr int W = BITS == 16 ? 8 : 16;
    typedef typename std::conditional<BITS == 16, uint16_t, uint8_t>::type E;
    constexpr int VS = D + 16 / (int)sizeof(E);
    constexpr int N = kBlockTokens * D / W;         // pieces of a block
    __shared__ __attribute__((aligned(16))) E s_x[2][kBlockTokens * VS];
    const int tid = threadIdx.x, nb = A.g.nb;
    const int head = blockIdx.x % A.c.heads, tb = blockIdx.x / A.c.heads % nb, r = blockIdx.x / A.c.heads / nb;
    kv::Req q = kv::request(A.B, A.c.page_shift, r);
    if (!q.ok) q.len = 0;                                           // only for numbering the rows
    const Span sp = span(q, tb);
    if (sp.lo >= sp.hi) return;
    const int64_t page = q.ok ? page_of(A.c, A.B, r, sp.base) : -1;
    const int t0 = sp.base & ((1 << A.c.page_shift) - 1);
    const int64_t chunk = page * A.c.heads + head;
    if (page >= 0) {
        const E *const ks = (const E *)A.c.k + chunk * chunk_elems<D, BITS>(A.c);
        const E *const vs = (const E *)A.c.v + chunk * chunk_elems<D, BITS>(A.c);
#pragma unroll 4
        for (int i = tid; i < N; i += TPB) {
            const int t = i / (16 * (D / W)) * 16 + i % 16, d = i / 64 % (D / (4 * W)) * 4 * W + i / 16 % 4 * W;
            const int sb = i / (64 * (D / 16)), vb = i / 64 % (D / 16), g = i / 16 % 4, dv = vb * 16 + i % 16;
            const int first = sb * 4 * W + g * 4;                   // v's positions: first + 16 jj + i
            const bool kin = t >= sp.lo && t < sp.hi, vin = first < sp.hi && first + 4 * W - 16 + 3 >= sp.lo;
            u32x4 a = {}, b = {};
            if (kin) a = *(const u32x4 *)(ks + kv::k_piece<D, W>(t0 + t, d));
            if (vin) b = *(const u32x4 *)(vs + kv::v_elem<D, W>(t0 + first, dv));
            if (kin) *(u32x4 *)(s_x[0] + t * VS + d) = a;
            if (vin) {
                struct { E e[W]; } x = __builtin_bit_cast(decltype(x), b);
#pragma unroll
                for (int j = 0; j < W; ++j) s_x[1][(first + j / 4 * 16 + j % 4) * VS + dv] = x.e[j];
            }
        }
        __syncthreads();
    }
    const int rows = sp.hi - sp.lo;
    for (int i = tid; i < 2 * rows * (D / 8); i += TPB) {
        const int which = i >= rows * (D / 8), at = which ? i - rows * (D / 8) : i;
        const int t = sp.lo + at / (D / 8), d = at % (D / 8) * 8;
        float x[8];
        if (page < 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(0x7fc00000u);
        } else if constexpr (BITS == 16) {
            Raw8<false> raw;
            raw.load(s_x[which], t * VS + d);
            raw.get(x);
        } else {
            const float s = (which ? A.c.vs : A.c.ks)[(chunk << A.c.page_shift) + t0 + t];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = s * (float)(int8_t)s_x[which][t * VS + d + e];
        }
        const int64_t to = (int64_t)(q.row0 + sp.base + t - q.len) * (which ? A.ldv : A.ldk) + head * D + d;
        if constexpr (F32) {
            float *const out = (float *)(which ? A.v : A.k) + to;
            *(f32x4 *)out = f32x4{x[0], x[1], x[2], x[3]};
            *(f32x4 *)(out + 4) = f32x4{x[4], x[5], x[6], x[7]};
        } else {
            *(u32x4 *)((uint16_t *)(which ? A.v : A.k) + to) = bf16_8(x);
        }
    }
}

// A request's path is taken, whole, if it starts at the root, rises strictly,
// stays below the nodes of a request and meets none but the cache's pages; else
// nothing is moved and nothing kept.  Every wave works it out by itself; `page`:
// the source's and the destination's of node path[lane].
__device__ __forceinline__ int kept_nodes(const KvCache &c, const AttnBatch &B, const int32_t *path,
                                          const int32_t *accept_len, int r, int32_t (&at)[2], int64_t (&page)[2]) {
    const int n = accept_len[r], lane = threadIdx.x & 63;
    const int32_t len = B.cache_len[r];
    bool bad = n < 1 || n > B.max_rows || len < 0 || (int64_t)len + B.max_rows > ((int64_t)B.max_pages << c.page_shift);
    if (bad) return 0;                                              // the same for all lanes
    if (lane < n) {
        const int32_t *p = path + (int64_t)r * B.max_rows;
        const int32_t node = p[lane];
        bad = lane == 0 ? node != 0 : node <= p[lane - 1] || node >= B.max_rows;
        at[0] = len + node;
        at[1] = len + lane;
    }
    if (__any(bad)) return 0;
    if (lane < n) {
        page[0] = page_of(c, B, r, at[0]);
        page[1] = page_of(c, B, r, at[1]);
        bad = page[0] < 0 || page[1] < 0;
    }
    return __any(bad) ? 0 : n;
}

__global__ __launch_bounds__(64) void new_len_kernel(const KvCache c, const AttnBatch B, const int32_t *path,
                                                     const int32_t *accept_len, int32_t *new_len) {
    int32_t at[2];
    int64_t page[2];
    const int r = blockIdx.x, n = kept_nodes(c, B, path, accept_len, r, at, page);
    if (threadIdx.x == 0) new_len[r] = B.cache_len[r] + n;
}

// Entry of node path[i] -> place i, for all i of a request, in one head of
// one cache.  Places are read before any is written (a place may hold a later
// node of the path).  Bound by the latency of path, page and entry, one after
// the other: 3.4-3.9 us for one cache, 7.2-10.3 for 64 of 4 requests.
template <int D, int BITS>
__global__ __launch_bounds__(TPB) void kv_commit_kernel(const CommitArgs A) {
    constexpr int W = BITS == 16 ? 8 : 16;
    typedef typename std::conditional<BITS == 16, uint16_t, uint8_t>::type E;
    __shared__ __attribute__((aligned(16))) E s_k[kMaxTree * D];
    __shared__ E s_v[kMaxTree * D];
    __shared__ float s_s[2][kMaxTree];
    __shared__ int64_t s_chunk[2][kMaxTree];                        // source and destination; -1: not moved
    __shared__ int32_t s_t[2][kMaxTree];
    const int tid = threadIdx.x, head = blockIdx.x, r = blockIdx.y;
    const CachePtrs C = A.caches[blockIdx.z];
    int32_t at[2];
    int64_t page[2];
    const int n = kept_nodes(A.c, A.B, A.path, A.accept_len, r, at, page);
    if (A.new_len != nullptr && head == 0 && blockIdx.z == 0 && tid == 0) A.new_len[r] = A.B.cache_len[r] + n;
    if (n <= 1) return;                                             // the root is in place
    if (tid < n) {
        const bool move = at[0] != at[1];
        s_chunk[0][tid] = move ? page[0] * A.c.heads + head : -1;
        s_chunk[1][tid] = page[1] * A.c.heads + head;
        s_t[0][tid] = at[0] & ((1 << A.c.page_shift) - 1);
        s_t[1][tid] = at[1] & ((1 << A.c.page_shift) - 1);
        if (BITS == 8 && move) {
            s_s[0][tid] = C.ks[(s_chunk[0][tid] << A.c.page_shift) + s_t[0][tid]];
            s_s[1][tid] = C.vs[(s_chunk[0][tid] << A.c.page_shift) + s_t[0][tid]];
        }
    }
    __syncthreads();
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        for (int i = tid; i < n * (D / W); i += TPB) {
            const int j = i / (D / W), d = i % (D / W) * W;
            if (s_chunk[0][j] < 0) continue;
            u32x4 *const p = (u32x4 *)((E *)C.k + s_chunk[pass][j] * chunk_elems<D, BITS>(A.c) +
                                       kv::k_piece<D, W>(s_t[pass][j], d));
            if (pass) *p = *(u32x4 *)(s_k + j * D + d); else *(u32x4 *)(s_k + j * D + d) = *p;
        }
        for (int i = tid; i < n * D; i += TPB) {
            const int j = i / D, d = i % D;
            if (s_chunk[0][j] < 0) continue;
            E *const p = (E *)C.v + s_chunk[pass][j] * chunk_elems<D, BITS>(A.c) + kv::v_elem<D, W>(s_t[pass][j], d);
            if (pass) *p = s_v[i]; else s_v[i] = *p;
        }
        if (!pass) __syncthreads();
    }
    if (BITS == 8 && tid < n && s_chunk[0][tid] >= 0) {
        C.ks[(s_chunk[1][tid] << A.c.page_shift) + s_t[1][tid]] = s_s[0][tid];
        C.vs[(s_chunk[1][tid] << A.c.page_shift) + s_t[1][tid]] = s_s[1][tid];
    }
}

// Calls f(std::integral_constant<int, D>, <int, BITS>) for the cache's format.
template <typename F>
void with_format(const KvCache &c, F f) {
    using std::integral_constant;
    const auto bits = [&](auto d) {
        if (c.bits == 16) f(d, integral_constant<int, 16>()); else f(d, integral_constant<int, 8>());
    };
    if (c.d == 64) bits(integral_constant<int, 64>());
    else if (c.d == 128) bits(integral_constant<int, 128>());
    else bits(integral_constant<int, 256>());
}

}  // namespace

hipError_t launch_append(const AppendArgs &A, hipStream_t s) {
    with_format(A.c, [&](auto d, auto bits) {
        if (A.f32)
            hipLaunchKernelGGL((append_kernel<d(), bits(), true>), dim3(A.g.grid), dim3(TPB), 0, s, A);
        else
            hipLaunchKernelGGL((append_kernel<d(), bits(), false>), dim3(A.g.grid), dim3(TPB), 0, s, A);
    });
    return hipGetLastError();
}

hipError_t launch_kv_read(const ReadArgs &A, hipStream_t s) {
    with_format(A.c, [&](auto d, auto bits) {
        if (A.f32)
            hipLaunchKernelGGL((kv_read_kernel<d(), bits(), true>), dim3(A.g.grid), dim3(TPB), 0, s, A);
        else
            hipLaunchKernelGGL((kv_read_kernel<d(), bits(), false>), dim3(A.g.grid), dim3(TPB), 0, s, A);
    });
    return hipGetLastError();
}

hipError_t launch_kv_commit(const CommitArgs &A, hipStream_t s) {
    with_format(A.c, [&](auto d, auto bits) {
        hipLaunchKernelGGL((kv_commit_kernel<d(), bits()>), dim3(A.c.heads, A.B.b, A.count), dim3(TPB), 0, s, A);
    });
    return hipGetLastError();
}

hipError_t launch_new_len(const CommitArgs &A, hipStream_t s) {
    hipLaunchKernelGGL(new_len_kernel, dim3(A.B.b), dim3(64), 0, s, A.c, A.B, A.path, A.accept_len, A.new_len);
    return hipGetLastError();
}

}  // namespace dspk
