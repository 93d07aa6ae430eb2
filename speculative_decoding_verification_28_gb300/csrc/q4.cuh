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
// fp32 rounding (a product corrected by its remainder) does not change the result: a tie
// is exact in fp32, and max |x| (11 bits at most) is otherwise at least 2^-12 of its value
// away from one.
__device__ __forceinline__ int q4_scale_byte(float amax)
{
    float f = amax * (1.0f / 7.0f);
    f = fmaf(fmaf(f, -7.0f, amax), 1.0f / 7.0f, f);
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

// About 1 / s, off by less than 2^-22 of it.
__device__ __forceinline__ float q4_reciprocal(float s)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return r;
}
// x / s to the nearest integer, ties to even, as a float; r about 1 / s.  A
// quotient below 8 is within 2^-19 of x r, and half way between integers or at least
// 2^-12 away from that (x has 11 bits at most, s four): 768 + x r, whose last bit is 2^-14,
// is exact where it is half way, and on the right side where it is not.  Adding 1.5 *
// 2^23 less 768 then rounds to integers.
__device__ __forceinline__ float q4_level(float x, float r)
{
    return __fsub_rn(__fadd_rn(fmaf(x, r, 768.0f), 12582912.0f - 768.0f), 12582912.0f);
}
// Four levels within -7 .. 7 as codes, in the low 16 bits: summed in fp32 with their
// place values, which is exact, and 2^23 + 0x8888 more, so that the integer pipe has
// one instruction for four.
__device__ __forceinline__ uint32_t q4_pack4(float a, float b, float c, float d)
{
    return __float_as_uint(__fadd_rn(fmaf(d, 4096.0f, fmaf(c, 256.0f, fmaf(b, 16.0f, a))), 8388608.0f + 34952.0f));
}

}  // namespace spec
