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
#include <type_traits>

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

// max(a, |v|, |w|) that keeps a NaN once it has met one.
__device__ __forceinline__ float abs_max(float a, float v, float w) {
    float m;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(fabsf(v)), "f"(fabsf(w)));
    return m;
}
// Two adjacent values of an array as the operand of a packed instruction
// (one issue for two fp32 operations, each rounded as usual): the kernels
// here are bound by instruction issue before they are bound by memory.
__device__ __forceinline__ float2 pair(const float* v) { return make_float2(v[0], v[1]); }
__device__ __forceinline__ void put(float* v, float2 p) {
    v[0] = p.x;
    v[1] = p.y;
}
__device__ __forceinline__ float2 twice(float v) { return make_float2(v, v); }

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

// Rounding v * inv to an integer by adding 1.5 * 2^23: the sum's low byte is
// the nearest integer (ties to even), for products below 2^22.  The product is
// rounded first, as the format says; the two may not be fused.  Codes need no
// clamp: |v| * inv exceeds 127 by a few roundings at most.  Conversion
// instructions run at an eighth of the add's rate, and two for each element
// were what bounded the activation's forward pass (16384 x 4096 gated bf16:
// 146 us with them).
constexpr float kIntBits = 12582912.f;
__device__ __forceinline__ uint32_t int_bits(float v, float inv) {
    return __float_as_uint(__fadd_rn(__fmul_rn(v, inv), kIntBits));
}

// Four codes in one word; inv = 0 gives codes 0 whatever v is (infinity * 0
// and NaN included).
template <int Q>
__device__ __forceinline__ uint32_t encode4(const float* v, float inv) {
    uint32_t c;
    const float2 a = __fmul2_rn(pair(v), twice(inv)), b = __fmul2_rn(pair(v + 2), twice(inv));
    if constexpr (Q == CT_Q_INT8) {
        // single additions: a packed one would be fused with the packed product
        const uint32_t lo = __byte_perm(__float_as_uint(__fadd_rn(a.x, kIntBits)), __float_as_uint(__fadd_rn(a.y, kIntBits)), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(__fadd_rn(b.x, kIntBits)), __float_as_uint(__fadd_rn(b.y, kIntBits)), 0x0040);
        c = __byte_perm(lo, hi, 0x5410);
    } else {
        c = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
            (uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16;
    }
    return inv == 0.f ? 0u : c;
}

template <int Q>
__device__ __forceinline__ uint8_t encode(float v, float inv) {
    if (inv == 0.f) return 0;
    if constexpr (Q == CT_Q_INT8) return (uint8_t)int_bits(v, inv);
    else return (uint8_t)__nv_cvt_float_to_fp8(v * inv, __NV_SATFINITE, __NV_E4M3);
}

template <int Q>
__device__ __forceinline__ float decode(uint8_t c) {
    if constexpr (Q == CT_Q_INT8) return (float)(int8_t)c;
    else return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3)));
}

// The four values of a word of codes (unscaled).  int8: a byte c + 128 put
// under the exponent of 2^23 is the number 2^23 + 128 + c, again without a
// conversion instruction.
template <int Q>
__device__ __forceinline__ void decode4(uint32_t c, float* v) {
    if constexpr (Q == CT_Q_INT8) {
        c ^= 0x80808080u;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(__byte_perm(c, 0x4b000000u, 0x7440 + i)) - 8388736.f;
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> (16 * i)), __NV_E4M3));
            const float2 f = __half22float2(h);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

// 1 / (1 + exp(-v)).  FAST (results that are rounded to 16 bits) takes the
// exponential and the reciprocal from the special-function unit as they are:
// relative error below 2^-21 + |v| 2^-24, an eighth of the instructions, and 0
// below v = -87.3, where the true value is below 1.2e-38.  fp32 results get a
// rounded quotient (silu of 16384 x 4096 gated 156 us; 150 with an approximate
// one, which is 0 from v = -87.3 on too and 2 units off elsewhere).
template <bool FAST>
__device__ __forceinline__ float sigmoid(float v) {
    if constexpr (FAST) {
        float e, r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
        return r;
    } else {
        return 1.f / (1.f + expf(-v));
    }
}

// Activation (ct_activation codes) and its derivative at v.
template <int A, bool FAST>
__device__ __forceinline__ float act_value(float v, float alpha) {
    if constexpr (A == 3) return v * sigmoid<FAST>(v);
    else if constexpr (A == 6) return sigmoid<FAST>(v);
    else return act_fixed<A>(v, alpha);
}

// Two at a time.
template <bool FAST>
__device__ __forceinline__ float2 sigmoid2(float2 v) {
    if constexpr (FAST) {
        const float2 t = __fmul2_rn(v, twice(-1.4426950408889634f));
        float2 e, r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
        e = __fadd2_rn(e, twice(1.f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
        return r;
    } else {
        return make_float2(sigmoid<false>(v.x), sigmoid<false>(v.y));
    }
}
template <int A, bool FAST>
__device__ __forceinline__ float2 act_value2(float2 v, float alpha) {
    if constexpr (A == 3) return __fmul2_rn(v, sigmoid2<FAST>(v));
    else if constexpr (A == 6) return sigmoid2<FAST>(v);
    else return make_float2(act_value<A, FAST>(v.x, alpha), act_value<A, FAST>(v.y, alpha));
}

template <int A, bool FAST>
__device__ __forceinline__ void act_both(float v, float alpha, float& f, float& slope) {
    if constexpr (A == 1) {
        f = v > 0.f ? v : 0.f;
        slope = v > 0.f ? 1.f : 0.f;
    } else if constexpr (A == 2) {
        f = v >= 0.f ? v : alpha * v;
        slope = v >= 0.f ? 1.f : alpha;
    } else if constexpr (A == 3) {
        const float s = sigmoid<FAST>(v);
        f = v * s;
        slope = fmaf(f, 1.f - s, s);
    } else if constexpr (A == 4) {
        const float cdf = 0.5f * (1.f + erff(v * 0.70710678118654752f));
        f = v * cdf;
        slope = fmaf(v * expf(-0.5f * v * v), 0.39894228040143268f, cdf);
    } else if constexpr (A == 5) {
        f = tanhf(v);
        slope = fmaf(-f, f, 1.f);
    } else if constexpr (A == 6) {
        f = sigmoid<FAST>(v);
        slope = f * (1.f - f);
    } else {
        f = v;
        slope = 1.f;
    }
}

template <int A, bool FAST>
__device__ __forceinline__ void act_both2(float2 v, float alpha, float2& f, float2& slope) {
    if constexpr (A == 3) {
        const float2 s = sigmoid2<FAST>(v);
        f = __fmul2_rn(v, s);
        slope = __ffma2_rn(f, __ffma2_rn(s, twice(-1.f), twice(1.f)), s);
    } else {
        act_both<A, FAST>(v.x, alpha, f.x, slope.x);
        act_both<A, FAST>(v.y, alpha, f.y, slope.y);
    }
}

// VEC consecutive elements of a row as one load or store of up to 16 bytes
// (VEC = 1: one element), widened to fp32.
template <typename T, int VEC>
struct Vec {
    static constexpr int kWords = VEC * (int)sizeof(T) >= 4 ? VEC * (int)sizeof(T) / 4 : 1;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const T* p) {
        if constexpr (VEC == 1) {
            if constexpr (sizeof(T) == 4) w[0] = *reinterpret_cast<const uint32_t*>(p);
            else w[0] = *reinterpret_cast<const unsigned short*>(p);
        } else {
            static_assert(sizeof(w) == 16, "one 16-byte access");
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (VEC == 1) {
            if constexpr (sizeof(T) == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
            else *reinterpret_cast<unsigned short*>(p) = (unsigned short)w[0];
        } else {
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else {
            const unsigned short b = (unsigned short)(w[i >> 1] >> ((i & 1) * 16));
            if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half(b));
            else return __uint_as_float((uint32_t)b << 16);
        }
    }
    // The largest |v| as the element type's own bits (ordered, NaN on top);
    // for 16-bit types two at a time.
    __device__ __forceinline__ uint32_t top_bits() const {
        uint32_t m = 0;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) m = max(m, w[i] & 0x7fffffffu);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
            m = max(m & 0xffffu, m >> 16);
        }
        return m;
    }
    // abs_bits of the fp32 value of such bits
    static __device__ __forceinline__ unsigned to_abs_bits(uint32_t m) {
        if constexpr (sizeof(T) == 4) return m;
        else if constexpr (std::is_same<T, __half>::value) return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
        else return m << 16;
    }
    // all VEC values at once, each rounded once
    __device__ __forceinline__ void set(const float (&v)[VEC]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[i] = __float_as_uint(v[i]);
        } else if constexpr (VEC == 1) {
            if constexpr (std::is_same<T, __half>::value) w[0] = __half_as_ushort(__float2half_rn(v[0]));
            else w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                if constexpr (std::is_same<T, __half>::value) {
                    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
        }
    }
};

// VEC codes written as one access.
template <int Q, int VEC>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&v)[VEC], float inv) {
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(p) = make_uint2(encode4<Q>(v, inv), encode4<Q>(v + 4, inv));
    else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(p) = encode4<Q>(v, inv);
    else *p = encode<Q>(v[0], inv);
}

// VEC (4 or 8) codes read as one access.
template <int VEC>
__device__ __forceinline__ void code_words(const uint8_t* p, uint32_t (&w)[VEC / 4]) {
    if constexpr (VEC == 8) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        w[0] = u.x;
        w[1] = u.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// Quotient and remainder by a divisor known to the host, for i < 2^31: m =
// floor(2^32 / d) + 1 gives the quotient or one more.  (d = 1: m = 0.)
struct Divider {
    unsigned d, m;
};
inline Divider divider(unsigned d) { return {d, d == 1 ? 0u : (unsigned)((1ull << 32) / d) + 1u}; }
__device__ __forceinline__ unsigned divide(unsigned i, Divider v, unsigned* rest) {
    if (v.m == 0) {
        *rest = 0;
        return i;
    }
    unsigned q = __umulhi(i, v.m);
    int r = (int)(i - q * v.d);
    if (r < 0) {
        --q;
        r += (int)v.d;
    }
    *rest = (unsigned)r;
    return q;
}

// Both halves of a word reduced at once (two 16-bit maxima in one).
__device__ __forceinline__ uint32_t lanes_max2(uint32_t v, int lanes) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
        if (o < lanes) v = __vmaxu2(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Maximum over `lanes` (a power of two) neighbouring lanes.
__device__ __forceinline__ unsigned lanes_max(unsigned v, int lanes) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
        if (o < lanes) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
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
