// The 4-bit cache row: 448 E2M1 codes in 14 groups of 32 with one UE8M0
// exponent each, and the 64 rope dims in bf16 (dsv4kv.h has the byte layout).
//
// The codes of 8 dims share a 32-bit word in the nibble order 0 2 4 6 1 3 5 7:
// nibbles i and i + 4 are dims 2i and 2i + 1, so one shift puts a neighbouring
// pair into the two halves of a bf16x2 word.  A code's value times 2^-126 is
// the bf16 whose exponent and mantissa fields are the code's (E2M1 0.5 becomes
// the bf16 subnormal 2^-127), so two exact packed multiplies, by 2^126 and by
// the group's scale, finish the conversion: an E2M1 value has two significant
// bits and every scale 2^(e - 127), e in [0, 254], is a bf16.  e = 255 marks a
// group that held a NaN or an infinity; its codes are 0 and 0 * inf reads NaN.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "bounds.cuh"
#include "convert.cuh"
#include "dsv4kv.h"
#include "fastdiv.h"

namespace dsv4 {
namespace {

constexpr uint32_t kFp4Slot = DSV4_FP4_SLOT_BYTES;
constexpr uint32_t kFp4Data = DSV4_FP4_DATA_BYTES;
constexpr uint32_t kFp4Codes = DSV4_NOPE_DIM / 2;

// Where a slot's bytes are.  block < num_blocks and off < block_size.
struct Fp4Row {
    const uint8_t *data;
    const uint8_t *scale;
};

__device__ __forceinline__ Fp4Row fp4_row(const uint8_t *cache, uint32_t block, uint32_t off,
                                          uint32_t block_size)
{
    const uint8_t *base = cache + uint64_t(block) * block_size * kFp4Slot;
    return Fp4Row{base + uint64_t(off) * kFp4Data,
                  base + uint64_t(block_size) * kFp4Data + uint64_t(off) * DSV4_FP4_SCALE_BYTES};
}

// 2^(e - 127) as a bf16 pattern in both halves (e = 255: infinity)
__device__ __forceinline__ uint32_t fp4_scale_bf16x2(uint32_t e)
{
    return (e == 0u ? 0x0040u : e << 7) * 0x00010001u;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// the 8 codes of a word as bf16 2^-126 times their values, in dim order
__device__ __forceinline__ uint4 fp4x8_small(uint32_t w)
{
    const auto pair = [](uint32_t sign, uint32_t rest) {
        return (sign & 0x80008000u) | (rest & 0x01C001C0u);
    };
    return make_uint4(pair(w << 12, w << 6), pair(w << 8, w << 2), pair(w << 4, w >> 2),
                      pair(w, w >> 6));
}

__device__ __forceinline__ uint4 mul_bf16x8(uint4 v, uint32_t k2)
{
    return make_uint4(mul_bf16x2(v.x, k2), mul_bf16x2(v.y, k2), mul_bf16x2(v.z, k2),
                      mul_bf16x2(v.w, k2));
}

// 8 bf16, what is not finite as a finite value
__device__ __forceinline__ uint4 finite_bf16x8(uint4 v)
{
    const auto one = [](uint32_t a) {
        // the lesser magnitude, with a's sign; of a NaN and a number the number
        asm("min.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(0x7F7F7F7Fu));
        return a;
    };
    return make_uint4(one(v.x), one(v.y), one(v.z), one(v.w));
}

// a + 0 * v over the 8 bf16 of v: what was 0 stays 0 unless a value is not finite
__device__ __forceinline__ uint32_t zero_of_bf16x8(uint4 v, uint32_t a)
{
    const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(a) : "r"(words[i]), "r"(0u));
    return a;
}

// the 8 codes of a word times the group's scale -> 8 bf16 in dim order, exact
__device__ __forceinline__ uint4 fp4x8_to_bf16(uint32_t w, uint32_t scale2)
{
    return mul_bf16x8(mul_bf16x8(fp4x8_small(w), 0x7E807E80u), scale2);  // by 2^126 first
}

// As matrix operands the rows are held times 2^-80: then 2^126 and the scale are one
// factor, 2^(e - 81), a bf16 for e <= 208 (values to 2^83; what stands above, e = 255
// among it, is `above`: infinite, or 0 where the row is marked instead).  What becomes
// subnormal was below 2^-46, far under the fp32 rounding of any sum with a normalised
// row.  Products take the 2^80 back in fp32.
constexpr float kOperandUnit = 0x1p80f;

constexpr uint32_t kOperandTop = 208u;

__device__ __forceinline__ uint32_t fp4_operand_scale(uint32_t e, uint32_t above)
{
    return (e > kOperandTop ? above : (e + 46u) << 7) * 0x00010001u;
}

// whether one of a row's 14 exponents is above kOperandTop
__device__ __forceinline__ bool fp4_row_above(uint4 scales)
{
    const uint32_t top = __vmaxu4(__vmaxu4(scales.x, scales.y),
                                  __vmaxu4(scales.z, scales.w & 0xFFFFu));
    return __vcmpgtu4(top, kOperandTop * 0x01010101u) != 0u;
}

constexpr uint32_t kRopeToOperand = 0x17801780u;  // bf16x2 (2^-80, 2^-80)

}  // namespace
}  // namespace dsv4
