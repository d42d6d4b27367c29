// ct_rows.cuh -- what the row operators (norm, 8-bit checkpoints, checkpointed
// activation) share: the 8-bit group format, activation slopes, reductions.
//
// The 8-bit format.  A row of `cols` values is cut into groups of `group`
// consecutive values (the last one may be shorter); each group has one fp32
// scale = amax / top (top = 127 for int8, 448 for e4m3), computed as
// amax * (1 / top), and codes = round(v * (1 / scale)).  Two kinds of groups
// are exceptions: one whose scale would be below the smallest normal fp32
// number gets scale 0 and codes 0 (its reciprocal would overflow), and one
// that holds an infinity or a NaN gets scale NaN and codes 0, so that the
// whole group reads back as NaN instead of as wrong finite values.
#pragma once

#include <cstdint>

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "ct.h"
#include "ct_types.cuh"

namespace ct {
namespace rows {

constexpr float kInvTopInt8 = 1.0f / 127.0f;
constexpr float kInvTopE4m3 = 1.0f / 448.0f;
constexpr unsigned kInfBits = 0x7f800000u;   // |v| at or above: infinity or NaN
constexpr float kMinNormal = 1.17549435e-38f;

// |v| as an unsigned number: ordered like |v|, with infinity and then NaN on
// top, so that one integer maximum finds both the largest magnitude and
// whether anything is not finite (fmaxf would drop a NaN).
__device__ __forceinline__ unsigned abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Scale and reciprocal scale of a group from the maximum of its abs_bits.
// Q: CT_Q_INT8 or CT_Q_E4M3.  inv = 0 marks a group whose codes are all 0.
template <int Q>
__device__ __forceinline__ void group_scale(unsigned amax_bits, float& scale, float& inv) {
    scale = __uint_as_float(amax_bits) * (Q == CT_Q_INT8 ? kInvTopInt8 : kInvTopE4m3);
    inv = 0.f;
    if (amax_bits >= kInfBits) scale = __uint_as_float(0x7fc00000u);
    else if (scale < kMinNormal) scale = 0.f;
    else inv = __frcp_rn(scale);
}

// One code.  With inv = 0 the code is 0 whatever v is (inf * 0 and NaN
// included).
template <int Q>
__device__ __forceinline__ uint8_t encode(float v, float inv) {
    if (inv == 0.f) return 0;
    if constexpr (Q == CT_Q_INT8) {
        const int q = __float2int_rn(v * inv);
        return (uint8_t)(int8_t)max(-127, min(127, q));
    } else {
        return (uint8_t)__nv_cvt_float_to_fp8(v * inv, __NV_SATFINITE, __NV_E4M3);
    }
}

template <int Q>
__device__ __forceinline__ float decode(uint8_t c) {
    if constexpr (Q == CT_Q_INT8) return (float)(int8_t)c;
    else return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3)));
}

// Derivative of act_fixed<A> (ct_types.cuh) at v.
template <int A>
__device__ __forceinline__ float act_slope(float v, float alpha) {
    if constexpr (A == 1) return v > 0.f ? 1.f : 0.f;
    else if constexpr (A == 2) return v >= 0.f ? 1.f : alpha;
    else if constexpr (A == 3) {
        const float s = 1.f / (1.f + expf(-v));
        return s * (1.f + v * (1.f - s));
    } else if constexpr (A == 4) {
        return 0.5f * (1.f + erff(v * 0.70710678118654752f)) + v * expf(-0.5f * v * v) * 0.39894228040143268f;
    } else if constexpr (A == 5) {
        const float t = tanhf(v);
        return 1.f - t * t;
    } else if constexpr (A == 6) {
        const float s = 1.f / (1.f + expf(-v));
        return s * (1.f - s);
    } else return 1.f;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the block, the same value in every thread; `part` holds 32 floats.
// A fixed order, so a result never depends on scheduling.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float* part) {
    v = warp_sum(v);
    if constexpr (THREADS == 32) return v;
    __syncthreads();  // an earlier sum may still be being read
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) s += part[w];
    return s;
}

}  // namespace rows
}  // namespace ct
