// fp8b_quant.cu -- block-scaled fp8 quantisation, alone and behind the
// residual addition and RMS norm of a transformer layer.
//
// Quantisation of a block X (one row x 128 columns, or 128 x 128):
//   s = max|X| / 448,  c = e4m3(x * (1 / s)), both in fp32;  a value is then c * s.
// Norm: r[t] = x[t] + sum_j w[t,j] delta[inv[t,j]] (a layer's combine, in slot
//   order) or x[t] + delta[t];  y[t,i] = r[t,i] g[i] / sqrt(mean_i r[t,i]^2 + eps);
//   r goes to the residual stream, y to bf16 (the router's input) and to codes.
//   The norm takes r as summed in fp32, before any rounding to the stream's type.
// Both are bound by memory: every value is read once into registers (16 bytes
// a load or more), reduced there, and written once.
#include "fp8b.h"
#include "kernels.h"

namespace moe {
namespace fp8b {

__device__ __forceinline__ void store8(float *p, const float (&v)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Largest magnitude (mag_bits) of 16 neighbouring lanes: one 1 x 128 block at
// 8 values per lane.
__device__ __forceinline__ uint32_t max16(uint32_t m)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}
__device__ __forceinline__ uint32_t max8(const float (&v)[8])
{
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, mag_bits(v[i]));
    return m;
}
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float f)
{
    return make_uint2(encode4(v[0], v[1], v[2], v[3], f), encode4(v[4], v[5], v[6], v[7], f));
}

// Eight values as loaded (bf16 stays packed: half the registers, and the
// maximum two values an instruction).
template <typename XT> struct Raw8;
template <> struct Raw8<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = __ldg(reinterpret_cast<const uint4 *>(p));
        b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    }
    __device__ __forceinline__ uint32_t max_bits() const
    {
        float v[8];
        get(v);
        return max8(v);
    }
};
template <> struct Raw8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[2 * i] = bf16lo(w[i]); v[2 * i + 1] = bf16hi(w[i]); }
    }
    __device__ __forceinline__ uint32_t max_bits() const
    {
        const uint32_t k = 0x7fff7fffu;
        const uint32_t m = __vmaxu2(__vmaxu2(a.x & k, a.y & k), __vmaxu2(a.z & k, a.w & k));
        return max(m << 16, m & 0xffff0000u);
    }
};

// ------------------------------------------------------------- quantisation
constexpr int kRowThreads = 256, kRowUnroll = 4;

// One row x 128 columns per half warp; kRowUnroll blocks in flight per half warp.
template <typename XT>
__global__ void __launch_bounds__(kRowThreads)
quant_rows_kernel(const XT *__restrict__ x, long long rows, int cols, long long ldx, int nblk,
                  uint8_t *__restrict__ codes, float *__restrict__ scales)
{
    pdl_enter();
    const int l16 = threadIdx.x & 15;
    const long long total = rows * nblk;
    const long long first = ((long long)blockIdx.x * kRowThreads + threadIdx.x) / 16;
    const long long step = (long long)gridDim.x * (kRowThreads / 16);
    // (every lane of a warp takes the same number of turns: the shuffles are warp-wide)
    const long long turns = (total + step * kRowUnroll - 1) / (step * kRowUnroll);
    for (long long turn = 0; turn < turns; ++turn) {
        Raw8<XT> c[kRowUnroll];
        long long row[kRowUnroll];
        int col[kRowUnroll], blk[kRowUnroll];
        bool in[kRowUnroll];
#pragma unroll
        for (int u = 0; u < kRowUnroll; ++u) {
            const long long b = first + (turn * kRowUnroll + u) * step;
            row[u] = b / nblk;
            blk[u] = (int)(b - row[u] * nblk);
            col[u] = blk[u] * kBlock + l16 * 8;
            in[u] = b < total && col[u] < cols;
            if (in[u]) c[u].load(x + row[u] * ldx + col[u]);
            else c[u].zero();
        }
#pragma unroll
        for (int u = 0; u < kRowUnroll; ++u) {
            const float s = block_scale(max16(c[u].max_bits()));
            if (!in[u]) continue;
            float v[8];
            c[u].get(v);
            *reinterpret_cast<uint2 *>(codes + row[u] * cols + col[u]) = encode8(v, code_factor(s));
            if (l16 == 0) scales[row[u] * nblk + blk[u]] = s;
        }
    }
}

constexpr int kTileThreads = 256, kTileChunks = kBlock * kBlock / 8 / kTileThreads;

// One 128 x 128 block per CTA, held in registers as loaded (8 chunks of 8
// values a thread).
template <typename XT>
__global__ void __launch_bounds__(kTileThreads)
quant_tiles_kernel(const XT *__restrict__ x, int rows, int cols, long long ldx, int nr, int nc,
                   uint8_t *__restrict__ codes, float *__restrict__ scales)
{
    pdl_enter();
    __shared__ uint32_t part[kTileThreads / 32];
    const long long tile = blockIdx.x;
    const long long band = tile / nc;                 // (batch, row block)
    const int bc = (int)(tile - band * nc);
    const long long b = band / nr;
    const int r0 = (int)(band - b * nr) * kBlock;
    const int col = bc * kBlock + (threadIdx.x & 15) * 8;
    Raw8<XT> c[kTileChunks];
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < kTileChunks; ++i) {
        const int r = r0 + (threadIdx.x >> 4) + i * (kTileThreads / 16);
        if (r < rows && col < cols) c[i].load(x + (b * rows + r) * ldx + col);
        else c[i].zero();
    }
#pragma unroll
    for (int i = 0; i < kTileChunks; ++i) m = max(m, c[i].max_bits());
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTileThreads / 32; ++w) m = max(m, part[w]);
    const float s = block_scale(m), f = code_factor(s);
    if (threadIdx.x == 0) scales[tile] = s;
#pragma unroll
    for (int i = 0; i < kTileChunks; ++i) {
        const int r = r0 + (threadIdx.x >> 4) + i * (kTileThreads / 16);
        float v[8];
        c[i].get(v);
        if (r < rows && col < cols)
            *reinterpret_cast<uint2 *>(codes + (b * rows + r) * cols + col) = encode8(v, f);
    }
}

// --------------------------------------------------------------------- norm
constexpr int kNormMaxThreads = 512, kNormMaxChunks = 4;
constexpr int kNormMaxWidth = kNormMaxThreads * kNormMaxChunks * 8;   // 16384

struct NormArgs {
    const void *x, *delta, *weight;
    const float *topk_w;
    const int32_t *inv;
    long long ldx, ldd;
    int T, d, k, delta_rows, weight_bf16, nblk;
    float eps;
    void *resid;
    __nv_bfloat16 *normed;
    uint8_t *codes;
    float *scales;
};

// One row per CTA, NV chunks of 8 values a thread, all in registers.  DT: the
// added rows' type (int: nothing is added).
template <typename XT, typename DT, int NV>
__global__ void __launch_bounds__(kNormMaxThreads, NV == 1 ? 4 : 1)   // (NV 1: 32 registers, 2048 threads an SM)
norm_kernel(const NormArgs a)
{
    pdl_enter();
    __shared__ float part[kNormMaxThreads / 32];
    constexpr bool kAdds = !std::is_same<DT, int>::value;
    const long long t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
    Chunk8 r[NV];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (threadIdx.x + j * blockDim.x) * 8;
        if (col < a.d) load8(static_cast<const XT *>(a.x) + t * a.ldx + col, r[j]);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) r[j].v[i] = 0.f;
    }
    if constexpr (kAdds) {
        const DT *delta = static_cast<const DT *>(a.delta);
        const int slots = a.k ? a.k : 1;
#pragma unroll 2
        for (int q = 0; q < slots; ++q) {
            // a slot whose grouped row is out of range (an expert id the
            // grouping left out) adds nothing
            const long long at = a.k ? (long long)__ldg(a.inv + t * a.k + q) : t;
            const float w = a.k ? __ldg(a.topk_w + t * a.k + q) : 1.f;
            if (at < 0 || at >= a.delta_rows) continue;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int col = (threadIdx.x + j * blockDim.x) * 8;
                if (col < a.d) {
                    Chunk8 y;
                    load8(delta + at * a.ldd + col, y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) r[j].v[i] = fmaf(w, y.v[i], r[j].v[i]);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (threadIdx.x + j * blockDim.x) * 8;
        if (kAdds && a.resid && col < a.d) store8(static_cast<XT *>(a.resid) + t * a.d + col, r[j].v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(r[j].v[i], r[j].v[i], sum);
    }
    sum = warp_sum(sum);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    sum = warp_sum(lane < nwarps ? part[lane] : 0.f);
    const float rs = 1.0f / sqrtf(sum / (float)a.d + a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (threadIdx.x + j * blockDim.x) * 8;
        const bool in = col < a.d;
        // y = z * rs with z = r * g
        if (in) {
            Chunk8 g;
            if (a.weight_bf16) load8(static_cast<const __nv_bfloat16 *>(a.weight) + col, g);
            else load8(static_cast<const float *>(a.weight) + col, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) r[j].v[i] *= g.v[i];
            if (a.normed) {
#pragma unroll
                for (int i = 0; i < 8; ++i) g.v[i] = r[j].v[i] * rs;
                store8(a.normed + t * a.d + col, g.v);
            }
        }
        const uint32_t zbits = max16(max8(r[j].v));
        if (in) {
            // The codes are those of y / s = 448 z / max|z|: the root and its
            // rounding cancel, which leaves the roundings of z, of 448 / max|z| and
            // of their product.  Where max|z| is so small that its factor could
            // overflow, z is scaled by rs first.
            const float zmax = __uint_as_float(zbits), ymax = zmax * rs;
            const float s = block_scale(zbits >= kInfBits ? zbits : mag_bits(ymax));
            const bool tiny = zmax < 0x1p-100f;
            const float f = s > 0.f ? kFp8Max / (tiny ? ymax : zmax) : s;   // (s = 0: zero codes, NaN: NaN)
            if (tiny) {
#pragma unroll
                for (int i = 0; i < 8; ++i) r[j].v[i] *= rs;
            }
            *reinterpret_cast<uint2 *>(a.codes + t * a.d + col) = encode8(r[j].v, f);
            if ((threadIdx.x & 15) == 0) a.scales[t * a.nblk + col / kBlock] = s;
        }
    }
}

template <typename XT, typename DT>
cudaError_t launch_norm(const NormArgs &a, cudaStream_t stream)
{
    // as many threads as chunks, up to 512; then 2 or 4 chunks a thread
    const int chunks = a.d / 8;
    const int nv = chunks <= kNormMaxThreads ? 1 : chunks <= 2 * kNormMaxThreads ? 2 : 4;
    const int threads = (int)align_up((size_t)ceil_div(chunks, nv), 32);
    const dim3 grid((unsigned)a.T), block(threads);
    if (nv == 1) return launch_pdl(norm_kernel<XT, DT, 1>, grid, block, 0, stream, a);
    if (nv == 2) return launch_pdl(norm_kernel<XT, DT, 2>, grid, block, 0, stream, a);
    return launch_pdl(norm_kernel<XT, DT, 4>, grid, block, 0, stream, a);
}
template <typename XT>
cudaError_t launch_norm_delta(const NormArgs &a, bool adds, int delta_dt, cudaStream_t stream)
{
    if (!adds) return launch_norm<XT, int>(a, stream);
    if (delta_dt == MOE_F32) return launch_norm<XT, float>(a, stream);
    return launch_norm<XT, __nv_bfloat16>(a, stream);
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool float_ok(int dt) { return dt == MOE_F32 || dt == MOE_BF16; }

}  // namespace fp8b
}  // namespace moe

using namespace moe;
using namespace moe::fp8b;

extern "C" {

moe_status moe_quant_fp8b(const void *x, moe_dtype x_dt, int batch, int rows, int cols, long long ldx,
                          int block_rows, void *codes, float *scales, moe_stream stream)
{
    if (batch < 0 || rows < 0 || cols <= 0 || cols % 16 || !float_ok(x_dt)) return MOE_ERR_INVALID_ARG;
    if (ldx < cols || ldx % 8) return MOE_ERR_INVALID_ARG;
    if (block_rows != 1 && block_rows != kBlock) return MOE_ERR_INVALID_ARG;
    if (batch == 0 || rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int nc = ceil_div(cols, kBlock);
    uint8_t *out = static_cast<uint8_t *>(codes);
    cudaError_t e;
    if (block_rows == 1) {
        const long long all = (long long)batch * rows;
        const long long per_cta = (kRowThreads / 16) * kRowUnroll;
        long long grid = (all * nc + per_cta - 1) / per_cta;
        if (grid > 0x7fffffffLL) grid = 0x7fffffffLL;   // (the kernel strides over the rest)
        e = x_dt == MOE_F32
                ? launch_pdl(quant_rows_kernel<float>, dim3((unsigned)grid), dim3(kRowThreads), 0, s,
                             static_cast<const float *>(x), all, cols, ldx, nc, out, scales)
                : launch_pdl(quant_rows_kernel<__nv_bfloat16>, dim3((unsigned)grid), dim3(kRowThreads), 0, s,
                             static_cast<const __nv_bfloat16 *>(x), all, cols, ldx, nc, out, scales);
    } else {
        const int nr = ceil_div(rows, kBlock);
        const long long tiles = (long long)batch * nr * nc;
        if (tiles > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
        e = x_dt == MOE_F32
                ? launch_pdl(quant_tiles_kernel<float>, dim3((unsigned)tiles), dim3(kTileThreads), 0, s,
                             static_cast<const float *>(x), rows, cols, ldx, nr, nc, out, scales)
                : launch_pdl(quant_tiles_kernel<__nv_bfloat16>, dim3((unsigned)tiles), dim3(kTileThreads), 0, s,
                             static_cast<const __nv_bfloat16 *>(x), rows, cols, ldx, nr, nc, out, scales);
    }
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_norm_fp8b(const void *x, moe_dtype x_dt, int T, int d, long long ldx, const void *delta,
                         moe_dtype delta_dt, int delta_rows, long long ldd, const float *topk_w,
                         const int32_t *inv, int k, const void *weight, moe_dtype weight_dt, float eps,
                         void *resid, void *normed, void *codes, float *scales, moe_stream stream)
{
    if (T < 0 || d <= 0 || d % 16 || k < 0 || !float_ok(x_dt) || !float_ok(weight_dt)) return MOE_ERR_INVALID_ARG;
    if (ldx < d || ldx % 8 || !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
    if (k > kMaxTopK || d > kNormMaxWidth) return MOE_ERR_UNSUPPORTED;
    const bool adds = delta || k > 0;   // (grouped rows may be none at all: delta NULL with delta_rows 0)
    if (k > 0 && !delta && delta_rows != 0) return MOE_ERR_INVALID_ARG;
    if (adds && (!float_ok(delta_dt) || ldd < d || ldd % 8 || delta_rows < 0)) return MOE_ERR_INVALID_ARG;
    if (adds && k == 0 && delta_rows < T) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!x || !weight || !codes || !scales || (k > 0 && (!topk_w || !inv))) return MOE_ERR_INVALID_ARG;
    if (adds && !resid) return MOE_ERR_INVALID_ARG;   // the sum would be lost
    if (!aligned(x, 16) || !aligned(delta, 16) || !aligned(weight, 16) || !aligned(resid, 16) ||
        !aligned(normed, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(topk_w, 4) || !aligned(inv, 4))
        return MOE_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = x; a.delta = delta; a.weight = weight; a.topk_w = topk_w; a.inv = inv;
    a.ldx = ldx; a.ldd = ldd; a.T = T; a.d = d; a.k = k; a.delta_rows = delta_rows;
    a.weight_bf16 = weight_dt == MOE_BF16; a.nblk = ceil_div(d, kBlock); a.eps = eps;
    a.resid = adds ? resid : nullptr;
    a.normed = static_cast<__nv_bfloat16 *>(normed);
    a.codes = static_cast<uint8_t *>(codes); a.scales = scales;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = x_dt == MOE_F32 ? launch_norm_delta<float>(a, adds, delta_dt, s)
                                          : launch_norm_delta<__nv_bfloat16>(a, adds, delta_dt, s);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
