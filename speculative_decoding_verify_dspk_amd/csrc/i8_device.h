// Device helpers of the 8-bit integer side.
#pragma once

#include <hip/hip_runtime.h>

#include "i8_internal.h"

namespace dspk {
namespace i8 {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint16_t to_bf16(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
__device__ __forceinline__ uint32_t to_bf16_pair(float lo, float hi) {
    return (uint32_t)to_bf16(lo) | ((uint32_t)to_bf16(hi) << 16);
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// A row's scale and the factor of its codes, from its largest magnitude (as
// bits, NaN on top): scale = top / 127, code = x * (127 / top) rounded half to even.
// held: false for a row that reads as NaN (scale NaN) or as zeros (below 4e-37,
// where 127 / top is no number), whose codes are zeros.
struct Step8 {
    float scale, inv;
    bool held;
};
__device__ __forceinline__ Step8 step8(uint32_t top) {
    Step8 s;
    const float t = __uint_as_float(top);
    s.inv = 127.f / t;
    s.held = top < 0x7f800000u && s.inv < __uint_as_float(0x7f800000u);
    s.scale = top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : s.held ? t / 127.f : 0.f;
    return s;
}
// Four codes.  1.5 * 2^23 added to the (rounded) product leaves it rounded half to even
// in the low bits, in two's complement.
__device__ __forceinline__ uint32_t codes8(float a, float b, float c, float d, const Step8 &s) {
#pragma clang fp contract(off)
    if (!s.held) return 0u;
    const float k = 12582912.f;
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(b * s.inv + k), __float_as_uint(a * s.inv + k), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(d * s.inv + k), __float_as_uint(c * s.inv + k), 0x04000c0cu);
    return lo | hi;
}

// A value of every lane and that of the lane a DPP control names, 0 where there is none.
template <int CTRL, int ROWS = 15>
__device__ __forceinline__ uint32_t from_lane(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 15, false);
}
// The largest value of the wave, to every lane: within rows of 16 lanes, then from row
// to row, by vector instructions alone (shuffles through LDS take ten times as long).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, from_lane<0x111>(v));
    v = max(v, from_lane<0x112>(v));
    v = max(v, from_lane<0x114>(v));
    v = max(v, from_lane<0x118>(v));
    v = max(v, from_lane<0x142, 10>(v));
    v = max(v, from_lane<0x143, 12>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// The sum of the wave, likewise.
__device__ __forceinline__ float wave_sum(float v) {
    v += __uint_as_float(from_lane<0x111>(__float_as_uint(v)));
    v += __uint_as_float(from_lane<0x112>(__float_as_uint(v)));
    v += __uint_as_float(from_lane<0x114>(__float_as_uint(v)));
    v += __uint_as_float(from_lane<0x118>(__float_as_uint(v)));
    v += __uint_as_float(from_lane<0x142, 10>(__float_as_uint(v)));
    v += __uint_as_float(from_lane<0x143, 12>(__float_as_uint(v)));
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// x / (1 + exp(-x)): exp as 2 to the rounded product with log2(e), times 1 + ln(2) times
// what that rounding and the constant's lost; the hardware's power and reciprocal are
// off by a step at most.  Where exp(-x) would pass fp32's largest number it counts as
// infinite.  (expf and a division: 1500 rows of 9728 28 us instead of 21.)
__device__ __forceinline__ float silu(float x) {
#pragma clang fp contract(off)
    const float y = fminf(fmaxf(x, -88.7f), 88.7f), hi = -1.44269504f, lo = -1.92596303e-8f;
    const float t = y * hi, r = fmaf(y, lo, fmaf(y, hi, -t));
    float e = __builtin_amdgcn_exp2f(t);
    e = fmaf(e, r * 0.693147181f, e);
    // a quarter of the denominator: its reciprocal is no subnormal number
    return x < -88.7f ? x * 0.f : .25f * x * __builtin_amdgcn_rcpf(fmaf(e, .25f, .25f));
}

// Data that other workgroups of the same launch read goes by device-scope accesses,
// which reach them without a cache flush; the writer waits for them before it counts
// itself in.
__device__ __forceinline__ void share(float *p, float a, float b) {
    __hip_atomic_store((unsigned long long *)p,
                       (unsigned long long)__float_as_uint(a) | (unsigned long long)__float_as_uint(b) << 32,
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void share(int32_t *p, int32_t a, int32_t b) {
    __hip_atomic_store((unsigned long long *)p, (unsigned long long)(uint32_t)a | (unsigned long long)(uint32_t)b << 32,
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ int2 shared2(const int32_t *p) {
    const unsigned long long v =
        __hip_atomic_load((unsigned long long *)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return make_int2((int32_t)(uint32_t)v, (int32_t)(uint32_t)(v >> 32));
}
__device__ __forceinline__ float2 shared2(const float *p) {
    const unsigned long long v =
        __hip_atomic_load((unsigned long long *)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}
// Counts a workgroup in after what its threads shared; true in the last of `of`.
// Every thread of the workgroup calls it.  The counter is left at zero by the last.
__device__ __forceinline__ bool last_to_arrive(uint32_t *counter, uint32_t of) {
    __shared__ uint32_t ticket;
    __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));          // vmcnt(0): this wave's data is performed
    __syncthreads();
    if (threadIdx.x == 0) {
        ticket = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (ticket == of - 1) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    return ticket == of - 1;
}

__device__ __forceinline__ i32x4 mfma64(i32x4 a, i32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// Four neighbouring columns of a row of y.
template <bool BF16>
__device__ __forceinline__ void store4(void *y, int64_t at, int32_t col, int32_t n, bool vec, const float (&v)[4]) {
    if (vec && col + 4 <= n) {
        if constexpr (BF16)
            *(u32x2 *)((uint16_t *)y + at) = u32x2{to_bf16_pair(v[0], v[1]), to_bf16_pair(v[2], v[3])};
        else
            *(f32x4 *)((float *)y + at) = f32x4{v[0], v[1], v[2], v[3]};
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (col + e >= n) break;
        if constexpr (BF16)
            ((uint16_t *)y)[at + e] = to_bf16(v[e]);
        else
            ((float *)y)[at + e] = v[e];
    }
}

}  // namespace i8
}  // namespace dspk
