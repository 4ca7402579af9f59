// fp8b.h -- shared pieces of the block-scaled fp8 operators (E4M3 codes, one
// fp32 scale per row and 128 columns, or per 128 x 128 block).
#pragma once

#include "common.cuh"

namespace moe {
namespace fp8b {

constexpr int kBlock = 128;          // columns (and weight rows) that share a scale
constexpr float kFp8Max = 448.0f;    // largest finite E4M3 value
constexpr uint32_t kInfBits = 0x7f800000u;

// |v| as bits: unsigned order is the order of magnitudes, with infinity above
// every finite value and NaN above infinity, so a maximum over these bits
// (unlike fmaxf) does not lose a NaN.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The scale of a block from the largest magnitude in it: amax / 448, and NaN
// for a block that holds an infinity or a NaN.
__device__ __forceinline__ float block_scale(uint32_t amax_bits)
{
    return amax_bits >= kInfBits ? __uint_as_float(0x7fffffffu) : __uint_as_float(amax_bits) / kFp8Max;
}

// Two values -> two E4M3 codes (low byte: the first), nearest, ties to even.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight values -> eight codes of v / s.  A true divide: the code of a value
// that lies on the border of two codes goes by the quotient itself, not by a
// rounded reciprocal (the quantising kernels are bound by memory).  s == 0
// (all values zero, or so small that amax / 448 underflows) gives zero codes;
// s = NaN gives NaN codes.
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float s)
{
    if (s == 0.f) return make_uint2(0u, 0u);
    uint2 o;
    o.x = e4m3x2(v[0] / s, v[1] / s) | (e4m3x2(v[2] / s, v[3] / s) << 16);
    o.y = e4m3x2(v[4] / s, v[5] / s) | (e4m3x2(v[6] / s, v[7] / s) << 16);
    return o;
}

}  // namespace fp8b
}  // namespace moe
