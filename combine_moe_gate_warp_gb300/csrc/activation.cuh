// activation.cuh -- the activations of the expert products, their slopes, and
// the 8-bit form of a saved layer (include/moe_experts.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "moe_experts.h"

namespace moe {

// The exponentials are __expf's, off by 2 + 1.18 |argument| steps of 2^-23
// relative to the value: below 2^-15 wherever fp32 holds the results here,
// which bf16 rounds by up to 2^-8.
__device__ __forceinline__ float logistic(float u) { return __fdividef(1.0f, 1.0f + __expf(-u)); }

// The normal distribution function Phi(u) = erfc(-u / sqrt 2) / 2 and
// exp(-u^2 / 2).  With z = |u| / sqrt 2 and t = 1 / (1 + z / 2),
//   erfc(z) exp(z^2) = t P(t),
// P the polynomial of degree 6 with the least largest error relative to the
// left side for |u| <= 13.5 (iteratively reweighted least squares): 2^-19.7.
// An absolute bound would not do: gelu below -5 is small, but it is a value
// of its own, and with formula 7.1.26 of Abramowitz and Stegun, 1.5e-7 at
// most, it was off by 0.4 % at -6 and 2 % at -10.  A third of erff's
// instructions, and both come from one exponential.
__device__ __forceinline__ float normal_cdf(float u, float &density)
{
    const float t = __fdividef(1.0f, fmaf(0.35355339059327376f, fabsf(u), 1.0f));
    float poly = fmaf(0.08903719f, t, -0.3596741f);
    poly = fmaf(poly, t, 0.3933407f);
    poly = fmaf(poly, t, 0.03497098f);
    poly = fmaf(poly, t, 0.2826016f);
    poly = fmaf(poly, t, 0.27737597f);
    poly = fmaf(poly, t, 0.28234646f);
    density = __expf(-0.5f * u * u);
    const float tail = 0.5f * poly * t * density;
    return u > 0.0f ? 1.0f - tail : tail;
}

__device__ __forceinline__ float act_value(float u, int act)
{
    float d;
    if (act == MOE_ACT_SILU) return u * logistic(u);
    if (act == MOE_ACT_GELU) return u * normal_cdf(u, d);
    return u;
}

// act'(u)
__device__ __forceinline__ float act_slope(float u, int act)
{
    if (act == MOE_ACT_SILU) {
        const float q = logistic(u);
        return q * (1.0f + u * (1.0f - q));
    }
    if (act == MOE_ACT_GELU) {
        float d;
        const float cdf = normal_cdf(u, d);
        return fmaf(u * d, 0.39894228040143268f, cdf);
    }
    return 1.0f;
}

// Scale byte of a saved block from the bit pattern of its largest magnitude
// (sign cleared): 127 + X, X the exponent of the smallest power of two with
// amax <= 448 * 2^X = 1.75 * 2^(X + 8); 255 for a NaN or an infinity.
__device__ __forceinline__ unsigned saved_byte(unsigned amax_bits)
{
    if (amax_bits >= 0x7F800000u) return 255u;
    // amax's exponent byte, one more where its fraction passes 1.75; a
    // subnormal has exponent byte 0 and lands below the clamp either way
    const int b = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (unsigned)max(b, 0);
}
// 1 / scale = 2^(127 - byte), exact (byte <= 247 for a finite amax)
__device__ __forceinline__ float saved_inverse(unsigned byte)
{
    return byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float((254u - byte) << 23);
}
// scale = 2^(byte - 127); 2^-127 is a subnormal
__device__ __forceinline__ float saved_scale(unsigned byte)
{
    return __uint_as_float(byte == 0u ? 0x400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

// lo in the low byte
__device__ __forceinline__ unsigned e4m3_pair(float lo, float hi)
{
    return (unsigned)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 e4m3_decode2(unsigned c)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xFFFFu), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
// four codes times their block's scale
__device__ __forceinline__ void saved_decode4(unsigned c, float scale, float *u)
{
    const float2 a = e4m3_decode2(c), b = e4m3_decode2(c >> 16);
    u[0] = a.x * scale;
    u[1] = a.y * scale;
    u[2] = b.x * scale;
    u[3] = b.y * scale;
}

__device__ __forceinline__ unsigned pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const unsigned *>(&v);
}
__device__ __forceinline__ uint2 pack_bf16x4(const float *v)
{
    return make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

}  // namespace moe
