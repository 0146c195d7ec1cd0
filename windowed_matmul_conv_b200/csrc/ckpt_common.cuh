// The 8-bit checkpoint code shared by the map and sequence kernels: the
// group's power-of-two step, and conversions of single values.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace wbmm {

constexpr uint32_t kAbsMask = 0x7fffffffu;
constexpr uint32_t kInfBits = 0x7f800000u;
constexpr uint32_t kExpBad = 255u;      // exponent byte of a group with a NaN or infinity
constexpr uint32_t kExpTop = 248u;      // the largest of the others, 2^121

// The larger of two bf16 magnitudes, pairwise; NaN (bits above infinity's)
// where either is.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Exponent byte of a group whose largest |x| has the fp32 bits `top` (NaN
// sorts above infinity, and both above every finite value).  127 steps have
// to reach |x| after rounding, i.e. |x| < 127.5 steps: with |x| = m 2^k,
// 1 <= m < 2, that is e = k - 6 for m < 127.5 / 64 = 1 + 0x7f0000 / 2^23 and
// one more above, which adding 0x010000 to the bits carries into the
// exponent.
__device__ __forceinline__ uint32_t group_exp(uint32_t top)
{
    if (top >= kInfBits)
        return kExpBad;
    const int e = (int)((top + 0x010000u) >> 23) - 6;
    return (uint32_t)(e < 1 ? 1 : e > (int)kExpTop ? (int)kExpTop : e);
}

// 2^(e - 127) for the exponent byte e; infinity for 255, so that code 128
// (0 * infinity) restores to NaN.
__device__ __forceinline__ float step_of(uint32_t e) { return __uint_as_float(e << 23); }

// 2^(127 - e), e <= 248 (0.0 for a bad group, whose values group_fix zeroes).
__device__ __forceinline__ float inv_step_of(uint32_t e)
{
    return e == kExpBad ? 0.0f : __uint_as_float((254u - e) << 23);
}

// For the groups with e >= kExpTop: zero in place of every value of a bad
// group, and at most 127 steps at the top of the range.
__device__ __forceinline__ float group_fix(float x, uint32_t e)
{
    const float top = 127.0f * __uint_as_float(kExpTop << 23);
    return e == kExpBad ? 0.0f : fminf(fmaxf(x, -top), top);
}

// rint(x / step) + 128 in the low byte, for |x| < 127.5 steps.  The product
// with a power of two is exact and adding 1.5 * 2^23 rounds it to an integer,
// ties to even.
__device__ __forceinline__ uint32_t quant_code(float x, float inv)
{
    return __float_as_uint(__fadd_rn(__fmul_rn(x, inv), 12583040.0f));
}

// Exact: 2^23 + code is a float, and its difference from 2^23 + 128 too.
__device__ __forceinline__ float code_value(uint32_t code, float step)
{
    return __fmul_rn(__fadd_rn(__uint_as_float(0x4b000000u | code), -8388736.0f), step);
}

}  // namespace wbmm
