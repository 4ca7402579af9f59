// fp8b_tc.cuh -- what the kernels of the block-scaled fp8 products share:
// parameters, tcgen05 kind::f8f6f4, tensor maps; the groups of a call and their tiles
// serve the int8 products too.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "fp8b.h"
#include "kernels.h"
#include "sm100.cuh"

namespace moe {
namespace tc {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();   // tc_gemm.cu
}
namespace fp8b {

using namespace sm100;

enum Mode { PRODUCT = 0, GATEUP = 1 };
enum Role { LOADS = 0, SUMS = 1 };   // whose first wait a test hook lets expire

struct Params {
    const float *x_s;         // [x_rows, KB]
    const float *w_s[2];      // [E, NB, KB] of W (PRODUCT) or W_gate, W_up
    const int32_t *offsets;   // [E+1], or NULL: one group of all rows
    const int32_t *perm_tok;  // [rows] (gathering)
    int E, rows, x_rows, K, N, KB, NB, n_tiles;
    void *out;                // PRODUCT: [rows, ldo] bf16 or fp32
    long long ldo;
    int out_f32, out_vec;     // out_vec: rows are multiples of 16 bytes apart, from a 16-byte boundary
    int out_tma;              // whole 32-row slices go out by TMA
    uint8_t *h_q;             // GATEUP: [rows, N] codes, [rows, NB] scales
    float *h_s;
    uint32_t *status;
    uint32_t expire_ns;       // > 0: the first wait of `expire_role` gives up after this long (test hook)
    int expire_role;
    int split;                // CTAs per cluster (fp8b_decode.cu)
};

// Instruction descriptor of tcgen05.mma kind::f8f6f4: fp32 accumulate, A and B
// E4M3 (format 0), both K-major, shape M x N.
constexpr uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
template <bool ACCUMULATE>
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "n"(ACCUMULATE ? 1 : 0)
        : "memory");
}
// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t is;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(is));
    return is != 0;
}
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
// Four rows y.x .. y.w of a 2-D tensor (box one row high), one below the other.
__device__ __forceinline__ void tma_gather4(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int4 y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w), "r"(smem_u32(bar))
        : "memory");
}
// mbar_wait, inline as a whole: across a call the compiler cannot keep the
// sums of the epilogue warps in the registers that setmaxnreg gives them.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                         unsigned long long timeout_ns = kTimeoutNs)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 255u) == 0) {
            if (*abort_flag) return false;
            if (globaltimer() - t0 > timeout_ns) return false;
        }
    }
}

// The test hook: whether this role's first wait is to give up.
__device__ __forceinline__ bool expires(const Params &p, Role role) { return p.expire_ns && p.expire_role == role; }

__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ float lo2(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
// two fp32 fused multiply-adds in one instruction, each rounded as fmaf is
__device__ __forceinline__ void fma2(uint64_t &acc, uint64_t a, uint64_t b)
{
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
// SwiGLU with the fast exponential and an approximate divide.  __expf(-g) is off
// by at most 2 + 1.173 |g| units in the last place, the sum, the divide (2 units)
// and the product by 3 more, so h is off by (5 + 1.18 |g|) 2^-23 of itself: 7e-7
// at g = 1, 1.3e-5 at g = -87, against the codes' 2^-4 (the scale, in fp32, is off
// by as much).  From g = -87.4 down the divisor is above 2^126, where __fdividef
// gives 0 (and infinity below -88.8, which gives 0 too): |silu(g)| < |g| 2^-126
// counts as 0.  g = -inf gives NaN, as -inf * 0 in the definition does.
__device__ __forceinline__ float swiglu(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The groups of a call and their tiles, in shared memory.
struct Groups {
    int total;   // tiles
    int off[kMaxExperts + 1], tile_start[kMaxExperts];
};
// Group bounds, kept inside [0, rows] whatever the array holds (every thread of
// the CTA; a barrier before scan_groups).
template <typename P> __device__ __forceinline__ void load_groups(Groups &g, const P &p)
{
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x)
        g.off[e] = p.offsets ? min(max(p.offsets[e], 0), p.rows) : e * p.rows;
}
// Exclusive scan of row tiles (of `rows_per_tile`) * column tiles over the
// experts, 8 to a lane (one warp).
template <typename P>
__device__ __forceinline__ void scan_groups(Groups &g, const P &p, int rows_per_tile, int lane)
{
    int local[8], sum = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = lane * 8 + j;
        int m = 0;
        if (e < p.E) m = (max(g.off[e + 1] - g.off[e], 0) + rows_per_tile - 1) / rows_per_tile;
        local[j] = m * p.n_tiles;
        sum += local[j];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    int run = incl - sum;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = lane * 8 + j;
        if (e < p.E) g.tile_start[e] = run;
        run += local[j];
    }
    if (lane == 31) g.total = incl;
}

struct Tile { int e, nt, row0, cnt; };   // expert, column tile, first grouped row, rows

// tile -> its expert, column tile and rows; within an expert the row tiles run
// fastest, so CTAs running at the same time share weight tiles through L2.
__device__ __forceinline__ Tile tile_at(const Groups &g, int E, int t, int rows_per_tile)
{
    int lo = 0, hi = E - 1;   // largest e with tile_start[e] <= t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (g.tile_start[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    const int local = t - g.tile_start[lo], m = (g.off[lo + 1] - g.off[lo] + rows_per_tile - 1) / rows_per_tile;
    Tile r;
    r.e = lo;
    r.nt = local / m;
    const int mt = local - r.nt * m;
    r.row0 = g.off[lo] + mt * rows_per_tile;
    r.cnt = min(rows_per_tile, g.off[lo + 1] - r.row0);
    return r;
}

// [n, rows, cols] codes (n = 0: [rows, cols]) with rows `ld` bytes apart, box
// {128 columns, box_rows}, 128-byte swizzle.
inline bool code_map(CUtensorMap *m, const void *base, int n, int rows, int cols, long long ld, uint32_t box_rows)
{
    auto enc = tc::encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)n};
    const cuuint64_t strides[2] = {(cuuint64_t)ld, (cuuint64_t)ld * (cuuint64_t)rows};
    const cuuint32_t box[3] = {(cuuint32_t)kBlock, box_rows, 1};
    const cuuint32_t one[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, n ? 3 : 2, const_cast<void *>(base), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// fp8b_decode.cu: the products of few rows, weights as the MMA's rows
bool decode_fits(const Params &p, int num_sms);
template <int MODE>
cudaError_t launch_decode(const void *x_q, long long ldx, const void *w0, const void *w1, Params p, int num_sms,
                          cudaStream_t stream);

}  // namespace fp8b
}  // namespace moe
