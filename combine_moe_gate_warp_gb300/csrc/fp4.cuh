// fp4.cuh -- rows of values in 4 bits (include/moe_route.h): 32 consecutive
// columns share a power of two, each value is an e2m1 code.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace moe {

// Scale byte of a block from the bf16 bits of its largest magnitude (sign
// cleared): 127 + X, X the smallest exponent with amax <= 6 * 2^X =
// 1.5 * 2^(X + 2); 255 for a NaN or an infinity.
__device__ __forceinline__ unsigned fp4_byte(unsigned amax)
{
    // amax's exponent byte, one more where its fraction passes 1.5; a
    // subnormal has exponent byte 0 and lands below the clamp either way
    const int b = (int)(amax >> 7) - 2 + ((amax & 0x7Fu) > 0x40u ? 1 : 0);
    return amax >= 0x7F80u ? 255u : (unsigned)max(b, 0);
}
// 2^(127 - byte), exact (byte <= 253 for a finite amax)
__device__ __forceinline__ float fp4_inverse(unsigned byte) { return __uint_as_float((254u - byte) << 23); }

// Eight values of magnitude 6 or less -> codes, value i in bits 4i ..; round
// to nearest, ties to the even code.
__device__ __forceinline__ unsigned fp4_encode8(const float *v)
{
    unsigned r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Two codes (bits 0-3 and 16-19 of c) as a pair of bf16.  A code's exponent
// and fraction bits, put where bf16 has them, are its value times 2^-126
// (subnormals too); two exact products bring it to scale: 2^126, and then
// 2^X, which alone may be a subnormal.
__device__ __forceinline__ unsigned fp4_decode2(unsigned c, unsigned scale)
{
    unsigned v = ((c & 0x00070007u) << 6) | ((c & 0x00080008u) << 12);
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(0x7E807E80u));
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(scale));
    return v;
}
// A scale byte as a pair of bf16: 2^(byte - 127); 2^-127 is a subnormal, 255 a NaN.
__device__ __forceinline__ unsigned fp4_scale2(unsigned byte)
{
    const unsigned s = byte == 0u ? 0x40u : byte == 255u ? 0x7FC0u : byte << 7;
    return s | (s << 16);
}

}  // namespace moe
