// fp8b.h -- shared pieces of the block-scaled fp8 operators (E4M3 codes, one
// fp32 scale per row and 128 columns, or per 128 x 128 block).
#pragma once

#include "common.cuh"

namespace moe {
namespace fp8b {

constexpr int kBlock = 128;          // columns (and weight rows) that share a scale
constexpr float kFp8Max = 448.0f;    // largest finite E4M3 value
constexpr float kMinNormal = 1.17549435e-38f;   // 2^-126
constexpr uint32_t kInfBits = 0x7f800000u;

// |v| as bits: unsigned order is the order of magnitudes, with infinity above
// every finite value and NaN above infinity, so a maximum over these bits
// (unlike fmaxf) does not lose a NaN.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The scale of a block from the largest magnitude in it: amax / 448; NaN for a
// block that holds an infinity or a NaN, 0 where amax / 448 is no normal number.
__device__ __forceinline__ float block_scale(uint32_t amax_bits)
{
    const float s = __uint_as_float(amax_bits) / kFp8Max;
    return amax_bits >= kInfBits ? __uint_as_float(0x7fffffffu) : s < kMinNormal ? 0.f : s;
}
// The factor that takes a block's values to codes, 1 / s (finite: s is normal);
// zero codes for s = 0, NaN codes for s = NaN.  One reciprocal a block and a
// product a value stand in for a divide a value: with the rounding of s their
// quotient is within 3 x 2^-24 of 448 x / max|x|, which moves a code only where
// that lies as close to the border of two.  bf16 values often lie on one exactly
// (448 x and max|x| have short significands): of 4.2 M normal values 5.0e-4 of the
// codes of 1 x 128 blocks (128 x 128: 2.4e-4) are a tie's other neighbour, not the
// even one, and no other code differs; of fp32 values about 1e-6.  Both neighbours
// of a tie are equally far, so the error is no larger.  x / s for every value, with
// s rounded, meets 9e-6 (2.7e-4) of them; (448 x) / max|x|, which would meet none
// in bf16, is a divide a value too.  (The divides made the quantisation of 92 M
// bf16 weights take 164 us, 4 times its memory traffic.)
__device__ __forceinline__ float code_factor(float s) { return s == 0.f ? 0.f : 1.0f / s; }

// Two values -> two E4M3 codes (low byte: the first), nearest, ties to even.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Four values times f -> four codes.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float f)
{
    return e4m3x2(a * f, b * f) | (e4m3x2(c * f, d * f) << 16);
}

}  // namespace fp8b
}  // namespace moe
