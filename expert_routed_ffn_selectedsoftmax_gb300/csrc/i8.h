// i8.h -- shared pieces of the 8-bit integer operators (int8 codes, one fp32 scale
// per row: a token of activations, an output channel of weights).
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace i8 {

enum Mode { PRODUCT = 0, GATEUP = 1 };
enum Role { LOADS = 0, CONVERT = 1, SUMS = 2 };   // whose first wait a test hook lets expire

// A product of the rows of every group with its expert's weights.
struct Params {
    const int8_t *x_q;        // [x_rows, K], rows ldx apart
    const float *x_s;         // [x_rows]
    const int8_t *w[2];       // [E, N, K] of W (PRODUCT) or W_gate, W_up
    const float *w_s[2];      // [E, N]
    const int32_t *offsets;   // [E+1], or NULL: one group of all rows
    const int32_t *perm_tok;  // [rows], or NULL: row r is x's row r
    long long ldx, ldo;
    int E, rows, x_rows, K, N;
    void *out;                // [rows, N] bf16 or fp32, rows ldo apart
    int out_f32, out_vec;     // out_vec: rows begin and end on 16-byte boundaries
    int n_tiles;              // column tiles (the tensor-core kernels)
    int split;                // CTAs of a cluster that share a reduction (i8_tc.cu)
    uint32_t *status;
    uint32_t expire_ns;       // > 0: the first wait of `expire_role` gives up after this long (test hook)
    int expire_role;
};

// Group e's rows, kept inside [0, rows] whatever the array holds.
__device__ __forceinline__ int group_bound(const Params &p, int e)
{
    return p.offsets ? min(max(__ldg(p.offsets + e), 0), p.rows) : e * p.rows;
}
// x's row of grouped row r (an index out of range reads row 0: its row is undefined).
__device__ __forceinline__ int source_row(const Params &p, int r)
{
    if (!p.perm_tok) return r;
    const int t = __ldg(p.perm_tok + r);
    return t >= 0 && t < p.x_rows ? t : 0;
}

// h = g / (1 + exp(-g)) u, from e = exp(-|g|): g / (1 + e), or g e / (1 + e) below zero, which is the
// larger of g and g e for either sign.  The divisor is between 1 and 2 and nothing overflows
// (with 1 + exp(-g) for a divisor, which __fdividef takes to 0 above 2^126, h was 0 from
// g = -87.4 down, whatever u).
//   fast      off by (5 + 1.18 |g|) 2^-23 of itself (__expf by 2 + 1.173 |g| units in the last
//             place, sum, divide and products by the rest), nothing beside a bf16 output's
//             half step of 2^-9
//   accurate  for fp32 outputs, 5 2^-23: expf and the reciprocal one unit each, the rest halves.
//             (A true divide is a call where its operands are extreme, and across a call the sums
//             do not stay in the registers that setmaxnreg gives.  A Newton step on the
//             reciprocal took up to 4 % of the tiled kernel's time, and the relative 2-norm
//             from 7.45e-8 to 7.35e-8 where g's own roundings leave 7.15e-8.)
// Below g = -87.3 e is less than the smallest normal number: off by (|g| + 2) 2^-149 |u| more.
// g = -inf gives NaN, as -inf * 0 in the definition does.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// 1 / d to one unit (of __fdividef's range nothing is needed).
__device__ __forceinline__ float reciprocal(float d)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    return r;
}
__device__ __forceinline__ float swiglu_of(float e, float g, float u) { return max_nan(g, g * e) * reciprocal(1.0f + e) * u; }
__device__ __forceinline__ float swiglu_fast(float g, float u) { return swiglu_of(__expf(-fabsf(g)), g, u); }
__device__ __forceinline__ float swiglu_accurate(float g, float u) { return swiglu_of(expf(-fabsf(g)), g, u); }

__device__ __forceinline__ void store_out(const Params &p, long long r, int n, float v)
{
    if (p.out_f32) static_cast<float *>(p.out)[r * p.ldo + n] = v;
    else static_cast<__nv_bfloat16 *>(p.out)[r * p.ldo + n] = __float2bfloat16_rn(v);
}

// i8_vector.cu -- products of a few rows per group on the CUDA cores
template <int MODE> cudaError_t launch_vector(const Params &p, cudaStream_t stream);

constexpr int kBlock = 128;    // columns of a block of a tensor-core kernel's reduction
constexpr int kMaxSplit = 8;   // CTAs of a cluster that share a reduction

// output channels of a tensor-core tile (its 128 weight rows are of W, or 64 of each of two)
constexpr int channels_of_tile(int mode) { return mode == GATEUP ? 64 : 128; }

// Most tiles of `tokens` rows there can be: an expert with r rows has (r - 1) / tokens + 1, so
// as many experts as possible with rows, and the rest of the rows in whole tiles.
inline long long most_tiles(int rows, int experts, int tokens)
{
    if (experts > rows) experts = rows;
    return (long long)(rows - experts) / tokens + experts;
}

// Few rows: CTAs that share a tile's reduction.  Tiles for fewer than half the SMs get a CTA
// for each SM, at most 8 a tile, where there are 8 blocks or more to share.
inline int split_of(long long tiles, int blocks, int sms)
{
    if (2 * tiles > sms || blocks < 8) return 1;
    const long long each = sms / tiles;
    return (int)(each < kMaxSplit ? each : kMaxSplit);
}

// i8_tc.cu -- the products on the tensor cores: tiles of 128 rows (their codes as fp16
// in `workspace`), or of few rows
size_t tiled_workspace(int rows, int K);
template <int MODE> cudaError_t launch_tiled(const Params &p, void *workspace, cudaStream_t stream);
// CTAs that share a 128-token tile's reduction: as many as all of them can run at the same
// time, 8, 4 or 2, where that takes more blocks off than the meeting costs (4.2 us; 0.335 a
// block).
template <int MODE> int split_of_tiled(long long tiles, int blocks);
template <int MODE> cudaError_t launch_few(const Params &p, cudaStream_t stream);

}  // namespace i8
}  // namespace moe
