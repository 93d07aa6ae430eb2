// q4.cuh -- the 4-bit format of a page pool (include/specverify.h) on the
// device: groups of 32 values with an 8-bit scale, codes of 4 bits.
//
// A scale byte b is the half with bits b << 7: no sign, five exponent and three
// mantissa bits.  A value (code - 8) * s has at most 7 significant bits, so it
// is exact in bf16 and fp16, and no product of a code and a scale ever rounds.
#pragma once

#include "spec_common.cuh"

namespace spec {

constexpr int kGroup = 32;         // values of a scale
constexpr int kTopScale = 223;     // 7680: seven times it is within fp16, and 1032 / 128 times it too
constexpr int kNanScale = 255;

// bytes of a token's codes and scales, and of a block of `page` tokens of a head
__host__ __device__ constexpr int q4_codes(int D) { return D / 2; }
__host__ __device__ constexpr int q4_scales(int D) { return D / kGroup; }
__host__ __device__ inline long long q4_block(int page, int D)
{
    return (long long)page * (q4_codes(D) + q4_scales(D));
}

// max |x| of a group -> the byte of max |x| / 7, rounded to even.  The quotient's
// fp32 rounding does not change the result: a tie is exact in fp32, and max |x|
// (11 bits at most) is otherwise at least 2^-12 of its value away from one.
__device__ __forceinline__ int q4_scale_byte(float amax)
{
    const float f = __fdiv_rn(amax, 7.0f);
    int b;
    if (f < 6.103515625e-05f) {  // 2^-14: steps of 2^-17
        b = __float2int_rn(f * 131072.0f);
    } else {
        const uint32_t u = __float_as_uint(f);
        b = (int)((u + 0x7FFFFu + (u >> 20 & 1u)) >> 20) - (112 << 3);
    }
    return max(1, min(b, kTopScale));
}
__device__ __forceinline__ float q4_scale(int byte) { return __half2float(__ushort_as_half((unsigned short)(byte << 7))); }

// x / s to the nearest code, ties to even.  q is the quotient rounded once
// (a product with the reciprocal r, corrected by its remainder), which is exact
// at ties; adding 1.5 * 2^23 + 8 rounds it to an integer in the low bits.
__device__ __forceinline__ uint32_t q4_code(float x, float s, float r)
{
    float q = x * r;
    q = fmaf(fmaf(-q, s, x), r, q);
    q = fminf(fmaxf(q, -7.0f), 7.0f);
    return __float_as_uint(q + 12582920.0f) & 15u;
}

}  // namespace spec
