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
// product a value stand in for a divide a value: their quotient is off by at
// most an ulp and a half of fp32, which moves a code only where the quotient
// lies that close to the border of two (the divides made the quantisation of
// 92 M bf16 weights take 164 us, 4 times its memory traffic).
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
