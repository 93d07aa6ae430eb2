// q4_expand.cuh -- codes of 4 bits to fp16 values on the device, shared by the
// attention kernels over pages.
//
// A nibble c under the bits of 1024 (or of 64, for a byte's upper one) is the half
// 1024 + c (64 + c); one multiply-add with the scale s' = s / 128 and -1032 s'
// (-72 s') gives (c - 8) s' exactly: 7 significant bits, s' >= 2^-24, and 1032 s'
// (11 bits) within fp16's range.  That is 2.3 instructions for two values
// (cvt of e2m1 pairs, with the scale's multiplication: 3.3).
#pragma once

#include "q4.cuh"

namespace spec {

constexpr float kQ4Units = 128.0f;  // what the expanded values are too small by

__device__ __forceinline__ uint32_t hfma2_bits(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// (a & b) | c in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// s' and its products, of a pair of scales: halves with bits byte << 7
struct Scale2 {
    uint32_t s, low, high;
    __device__ __forceinline__ explicit Scale2(uint32_t halves)
    {
        s = hmul2_bits(halves, 0x20002000u);  // 2^-7
        low = hmul2_bits(s, 0xE408E408u);     // -1032
        high = hmul2_bits(s, 0xD480D480u);    // -72
    }
};
// nibbles 0, 1, 2, 3 of both halves of w, as values
__device__ __forceinline__ void q4_expand(uint32_t w, const Scale2 &s, uint32_t *x)
{
    const uint32_t v = w >> 8;
    x[0] = hfma2_bits(and_or(w, 0x000F000Fu, 0x64006400u), s.s, s.low);
    x[1] = hfma2_bits(and_or(w, 0x00F000F0u, 0x54005400u), s.s, s.high);
    x[2] = hfma2_bits(and_or(v, 0x000F000Fu, 0x64006400u), s.s, s.low);
    x[3] = hfma2_bits(and_or(v, 0x00F000F0u, 0x54005400u), s.s, s.high);
}

// The same in bf16, in units of their own: under the bits of 128, 128 + c, times s
// and -136 s (8 significant bits).
struct Scale2Bf16 {
    uint32_t s, low;
    __device__ __forceinline__ explicit Scale2Bf16(uint32_t byte)
    {
        // bits byte << 4 are s * 2^-112
        const uint32_t raw = byte == kNanScale ? 0x7FC07FC0u : byte * 0x00100010u;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(s) : "r"(raw), "r"(0x77807780u));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(low) : "r"(s), "r"(0xC308C308u));
    }
};
__device__ __forceinline__ void q4_expand(uint32_t w, const Scale2Bf16 &s, uint32_t *x)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("fma.rn.bf16x2 %0, %1, %2, %3;"
            : "=r"(x[i])
            : "r"(and_or(w >> (4 * i), 0x000F000Fu, 0x43004300u)), "r"(s.s), "r"(s.low));
}

// The eight 16-bit values of a 16-byte word in the order in which a word of
// codes expands: (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ void pairs_of(const uint4 &x, uint32_t *p)
{
    p[0] = __byte_perm(x.x, x.z, 0x5410);
    p[1] = __byte_perm(x.x, x.z, 0x7632);
    p[2] = __byte_perm(x.y, x.w, 0x5410);
    p[3] = __byte_perm(x.y, x.w, 0x7632);
}

// A word's values as they come out -> in order.
__device__ __forceinline__ uint4 in_order(const uint32_t *x)
{
    return make_uint4(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410), __byte_perm(x[0], x[1], 0x7632),
                      __byte_perm(x[2], x[3], 0x7632));
}

// exponent e of the power of two that a bf16 row with largest magnitude `top`,
// 2^-64 at least, is held times in fp16: top goes to 2^8 .. 2^9.  What falls under
// fp16's steps is then less than 2^-32 of it, less than fp32 sums keep.  Smaller rows
// (subnormal ones among them) come times 2^64 first, kSmallRow: 2^e alone would be
// past fp32's range for them.
constexpr float kSmallRow = 18446744073709551616.0f;
__device__ __forceinline__ int q4_row_exponent(float top)
{
    return top > 0.0f && top <= 3.4e38f ? 8 - ((int)(__float_as_uint(top) >> 23) - 127) : 0;
}

}  // namespace spec
