// FP8 cache rows as matrix operands: 448 E4M3 codes in 7 blocks of 64 dims with a UE8M0
// exponent each, and 64 rope dims in bf16 (dsv4kv.h has the byte layout).
//
// An E4M3 code's exponent and mantissa fields, put where a bf16's low exponent bits and high
// mantissa bits are, read as 2^-120 times the code's value, subnormal codes included; an
// E4M3 value has four significant bits and a block's scale is a power of two, so one packed
// multiplication finishes the conversion exactly.  The rows are held times 2^-48: then the
// factor 2^120 * 2^(e - 127) * 2^-48 = 2^(e - 55) is a bf16 for e <= 182 (values below 2^64),
// and what becomes subnormal was below 2^-78, far under the fp32 rounding of any sum with
// a normalised row.  Products take the 2^48 back in fp32.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dsv4kv.h"

namespace dsv4 {
namespace {

constexpr float kFp8OperandUnit = 0x1p48f;
constexpr uint32_t kFp8OperandTop = 182u;            // the largest exponent byte that fits
constexpr uint32_t kFp8RopeToOperand = 0x27802780u;  // bf16x2 (2^-48, 2^-48)

__device__ __forceinline__ uint32_t mul_bf16x2_rn(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// 2^(e - 55) in both halves, for e <= kFp8OperandTop
__device__ __forceinline__ uint32_t fp8_operand_scale(uint32_t e)
{
    return ((e + 72u) << 7) * 0x00010001u;
}

// Four codes -> four bf16 of 2^-120 times their values.  A byte goes to the low half of 16
// bits under copies of its sign; shifted left by 4 and masked that is the sign at bit 15 and
// the seven other bits at 4..10 (what crosses from the lower half is masked off).
__device__ __forceinline__ uint2 e4m3x4_small(uint32_t w)
{
    uint32_t lo, hi;
    asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(lo) : "r"(w));
    asm("prmt.b32 %0, %1, 0, 0xb3a2;" : "=r"(hi) : "r"(w));
    return make_uint2((lo << 4) & 0x87f087f0u, (hi << 4) & 0x87f087f0u);
}

// 8 codes times a scale -> 8 bf16
__device__ __forceinline__ uint4 e4m3x8_scaled(uint32_t w0, uint32_t w1, uint32_t scale2)
{
    const uint2 a = e4m3x4_small(w0), b = e4m3x4_small(w1);
    return make_uint4(mul_bf16x2_rn(a.x, scale2), mul_bf16x2_rn(a.y, scale2),
                      mul_bf16x2_rn(b.x, scale2), mul_bf16x2_rn(b.y, scale2));
}

// nonzero if one of 16 codes is NaN (all seven bits under the sign set)
__device__ __forceinline__ uint32_t e4m3x16_nan(uint4 c)
{
    const auto one = [](uint32_t w) { return (~w & 0x7f7f7f7fu) - 0x01010101u; };
    return (one(c.x) | one(c.y) | one(c.z) | one(c.w)) & 0x80808080u;
}

__device__ __forceinline__ uint4 fp8_rope_operand(uint4 v)
{
    return make_uint4(mul_bf16x2_rn(v.x, kFp8RopeToOperand), mul_bf16x2_rn(v.y, kFp8RopeToOperand),
                      mul_bf16x2_rn(v.z, kFp8RopeToOperand), mul_bf16x2_rn(v.w, kFp8RopeToOperand));
}

// nonzero if one of 8 bf16 is not finite: 0 times it is NaN
__device__ __forceinline__ uint32_t bf16x8_not_finite(uint4 v)
{
    uint32_t a = 0u;
    const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(a) : "r"(words[i]), "r"(0u));
    return a & 0x7fff7fffu;
}

}  // namespace
}  // namespace dsv4
