// dispatch.cu -- rows on their way to the experts and back: dispatch (tokens into
// grouped order), combine (the experts' outputs back to tokens, weighted), and the
// backward pass of both.
//
//   dispatch           out[inv[t,j]] = x[t]
//     backward         dx[t] = sum_j g[inv[t,j]]
//   combine            out[t] = sum_j w[t,j] y[inv[t,j]]
//     backward         dy[inv[t,j]] = w[t,j] g[t],   dw[t,j] = sum_i g[t,i] y[inv[t,j],i]
//
// All of them go by tokens: a token's row is read (or written) once and its k
// grouped rows are found through inv, so each byte moves once and nothing needs an
// atomic.  A thread holds 8 columns of its token and asks for the k rows' at once.  What bounds them is memory.  Sums run over the
// slots in order, in fp32, and are rounded once.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace rows {

constexpr int kThreads = 256;
constexpr int V = 8;            // columns of a thread's chunk

// V columns of a thread.  VEC: neighbours, 16 bytes a load (or two).  Else, where rows do not
// lie on 16-byte boundaries, `step` apart, an element a load: the threads of a row still
// read neighbouring elements, and V loads are in flight.
template <typename T, bool VEC> struct Chunk;
template <typename T> struct Bits;
template <> struct Bits<float> {
    using Raw = uint32_t;
    __device__ static __forceinline__ float get(uint32_t r) { return __uint_as_float(r); }
    __device__ static __forceinline__ uint32_t put(float v) { return __float_as_uint(v); }
};
template <> struct Bits<__nv_bfloat16> {
    using Raw = uint16_t;
    __device__ static __forceinline__ float get(uint16_t r) { return __uint_as_float((uint32_t)r << 16); }
    __device__ static __forceinline__ uint16_t put(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
};
template <typename T> struct Chunk<T, false> {
    typename Bits<T>::Raw a[V];
    __device__ __forceinline__ void load(const T *p, int step, int left)
    {
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] = i * step < left ? __ldg(reinterpret_cast<const typename Bits<T>::Raw *>(p) + i * step) : 0;
    }
    __device__ __forceinline__ void store(T *p, int step, int left) const
    {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * step < left) reinterpret_cast<typename Bits<T>::Raw *>(p)[i * step] = a[i];
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] = 0;
    }
    __device__ __forceinline__ float get(int i) const { return Bits<T>::get(a[i]); }
    __device__ __forceinline__ void set(const float (&v)[V])
    {
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] = Bits<T>::put(v[i]);
    }
};
template <> struct Chunk<float, true> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float *p, int, int)
    {
        a = __ldg(reinterpret_cast<const uint4 *>(p));
        b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    }
    __device__ __forceinline__ void store(float *p, int, int) const
    {
        reinterpret_cast<uint4 *>(p)[0] = a;
        reinterpret_cast<uint4 *>(p)[1] = b;
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ float get(int i) const
    {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        return __uint_as_float(w[i]);
    }
    __device__ __forceinline__ void set(const float (&v)[V])
    {
        a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    }
};
template <> struct Chunk<__nv_bfloat16, true> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, int, int) { a = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void store(__nv_bfloat16 *p, int, int) const { *reinterpret_cast<uint4 *>(p) = a; }
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ float get(int i) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
        return (i & 1) ? bf16hi(w[i >> 1]) : bf16lo(w[i >> 1]);
    }
    __device__ __forceinline__ void set(const float (&v)[V])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        a = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

struct Args {
    const void *x;            // dispatch: [T, d]; combine: y [rows, d]
    const void *g;            // combine's backward: [T, d]
    const float *topk_w;      // [T, k], or NULL: weights 1
    const int32_t *inv;       // [T*k]
    void *out;
    float *dw;
    long long ldx, ldg, ldo;  // elements from row to row
    int T, k, rows, d;
    int col_blocks;           // CTAs along a row
    int lanes_log2;           // threads of a CTA along a row
};

// This thread's token and first column; a CTA holds kThreads >> lanes_log2 tokens, and a
// row's chunks are spread over col_blocks CTAs (a thread takes one chunk, so that a few
// tokens still fill the SMs).  Without VEC its columns lie 1 << lanes_log2 apart.
template <bool VEC> __device__ __forceinline__ bool place(const Args &a, long long &t, int &col)
{
    const int lanes = 1 << a.lanes_log2, lane = threadIdx.x & (lanes - 1);
    const long long tb = blockIdx.x / a.col_blocks;
    t = tb * (kThreads >> a.lanes_log2) + (threadIdx.x >> a.lanes_log2);
    col = (int)(blockIdx.x - tb * a.col_blocks) * (lanes * V) + (VEC ? lane * V : lane);
    return t < a.T && col < a.d;
}

template <typename XT, bool VEC>
__global__ void __launch_bounds__(kThreads)
scatter_rows_kernel(const Args a)
{
    pdl_enter();
    long long t;
    int col;
    if (!place<VEC>(a, t, col)) return;
    const int step = 1 << a.lanes_log2, left = a.d - col;
    Chunk<XT, VEC> c;
    c.load(static_cast<const XT *>(a.x) + t * a.ldx + col, step, left);
    XT *out = static_cast<XT *>(a.out) + col;
    const int32_t *inv = a.inv + t * a.k;
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {
        const int r = __ldg(inv + j);
        if (r >= 0 && r < a.rows) c.store(out + r * a.ldo, step, left);
    }
}

// WEIGHTED: combine; else dispatch's backward pass.
template <typename XT, typename OT, bool VEC, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads)
gather_sum_kernel(const Args a)
{
    pdl_enter();
    long long t;
    int col;
    if (!place<VEC>(a, t, col)) return;
    const int step = 1 << a.lanes_log2, left = a.d - col;
    const XT *x = static_cast<const XT *>(a.x) + col;
    const int32_t *inv = a.inv + t * a.k;
    const float *w = a.topk_w + t * a.k;
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.f;
    constexpr int U = VEC ? 4 : 2;   // rows asked for at once
    for (int j0 = 0; j0 < a.k; j0 += U) {
        Chunk<XT, VEC> c[U];
        float f[U];
        bool in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = j0 + u < a.k ? __ldg(inv + j0 + u) : -1;
            in[u] = r >= 0 && r < a.rows;
            f[u] = 1.f;
            if (in[u]) {
                c[u].load(x + r * a.ldx, step, left);
                if (WEIGHTED) f[u] = __ldg(w + j0 + u);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!in[u]) continue;   // (a slot without a row adds nothing, whatever its weight)
#pragma unroll
            for (int i = 0; i < V; ++i) sum[i] = WEIGHTED ? fmaf(f[u], c[u].get(i), sum[i]) : sum[i] + c[u].get(i);
        }
    }
    Chunk<OT, VEC> o;
    o.set(sum);
    o.store(static_cast<OT *>(a.out) + t * a.ldo + col, step, left);
}

// Combine's backward pass: a token to a group of `G` threads (a warp, or the CTA),
// which walk its chunks; each thread sums its part of every slot's product, and the
// parts meet in a fixed order (shuffles, then the warps in order).
template <typename XT, typename GT, bool VEC, int G>
__global__ void __launch_bounds__(kThreads)
combine_backward_kernel(const Args a)
{
    pdl_enter();
    __shared__ float part[kThreads / 32][kMaxTopK];
    const int lane = threadIdx.x & (G - 1);
    const long long t = (long long)blockIdx.x * (kThreads / G) + threadIdx.x / G;
    float dot[kMaxTopK];
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) dot[j] = 0.f;
    if (t < a.T) {
        const XT *y = static_cast<const XT *>(a.x);
        const GT *g = static_cast<const GT *>(a.g) + t * a.ldg;
        XT *dy = static_cast<XT *>(a.out);
        int r[kMaxTopK];
        float w[kMaxTopK];
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j) {
            r[j] = j < a.k ? __ldg(a.inv + t * a.k + j) : -1;
            if (r[j] >= a.rows) r[j] = -1;
            w[j] = j < a.k ? __ldg(a.topk_w + t * a.k + j) : 0.f;
        }
        constexpr int C = VEC ? 2 : 1;   // chunks in flight
        for (int base = 0; base < a.d; base += C * G * V) {
            Chunk<GT, VEC> c[C];
            int col[C];
#pragma unroll
            for (int q = 0; q < C; ++q) {
                col[q] = base + q * G * V + (VEC ? lane * V : lane);
                c[q].zero();
                if (col[q] < a.d) c[q].load(g + col[q], G, a.d - col[q]);
            }
            // (two rows at a time: their loads stand ahead of the stores)
#pragma unroll
            for (int j0 = 0; j0 < kMaxTopK; j0 += 2) {
                if (j0 >= a.k) break;
                Chunk<XT, VEC> v[C][2];
#pragma unroll
                for (int q = 0; q < C; ++q)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        v[q][u].zero();
                        if (r[j0 + u] >= 0 && a.dw && col[q] < a.d) v[q][u].load(y + r[j0 + u] * a.ldx + col[q], G, a.d - col[q]);
                    }
#pragma unroll
                for (int q = 0; q < C; ++q)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int j = j0 + u;
                        if (r[j] < 0 || col[q] >= a.d) continue;
                        float o[V];
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            dot[j] = fmaf(c[q].get(i), v[q][u].get(i), dot[j]);
                            o[i] = w[j] * c[q].get(i);
                        }
                        if (dy) {
                            Chunk<XT, VEC> s;
                            s.set(o);
                            s.store(dy + r[j] * a.ldo + col[q], G, a.d - col[q]);
                        }
                    }
            }
        }
    }
    if (!a.dw) return;   // (the whole grid)
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
        if (j >= a.k) break;
        dot[j] = warp_sum(dot[j]);
        if (G > 32 && lane % 32 == 0) part[threadIdx.x / 32][j] = dot[j];
        if (G == 32 && lane == 0 && t < a.T) a.dw[t * a.k + j] = dot[j];
    }
    if (G > 32) {
        __syncthreads();
        const int j = threadIdx.x & (G - 1);
        if (t < a.T && j < a.k) {
            float s = 0.f;
            for (int q = 0; q < G / 32; ++q) s += part[threadIdx.x / G * (G / 32) + q][j];
            a.dw[t * a.k + j] = s;
        }
    }
}

// ------------------------------------------------------------------- host
bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t size_of(int dt) { return dt == MOE_F32 ? 4 : 2; }
bool float_ok(int dt) { return dt == MOE_F32 || dt == MOE_BF16; }
// rows that V columns at a time can walk: both ends of a row on 16-byte boundaries
bool vectors(const void *p, long long ld, int d) { return d % V == 0 && ld % V == 0 && aligned(p, 16); }

// The sizes of a call; MOE_OK with *go = false for one without tokens.
moe_status check(int T, int k, int rows, int d, const int32_t *inv, bool *go)
{
    *go = false;
    if (T < 0 || k < 1 || rows < 0 || d <= 0) return MOE_ERR_INVALID_ARG;
    if (k > kMaxTopK) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (T > INT32_MAX / kMaxTopK) return MOE_ERR_UNSUPPORTED;
    if (!inv || !aligned(inv, 4)) return MOE_ERR_INVALID_ARG;
    *go = true;
    return MOE_OK;
}
// A matrix's pointer and row distance (`may_be_empty`: without rows it may be NULL).
bool matrix_ok(const void *p, moe_dtype dt, long long ld, int d, bool may_be_empty)
{
    return float_ok(dt) && ld >= d && (p || may_be_empty) && aligned(p, size_of(dt));
}

// grid of a kernel whose threads take a chunk each
bool lay_out(Args &a, dim3 *grid)
{
    const int chunks = ceil_div(a.d, V);
    a.lanes_log2 = 5;
    while (a.lanes_log2 < 8 && (1 << a.lanes_log2) < chunks) ++a.lanes_log2;
    a.col_blocks = ceil_div(chunks, 1 << a.lanes_log2);
    const int per = kThreads >> a.lanes_log2;
    const long long ctas = ((long long)a.T + per - 1) / per * a.col_blocks;
    *grid = dim3((unsigned)ctas);
    return ctas <= 0x7fffffffLL;
}

template <typename F> moe_status launched(F launch)
{
    return launch() == cudaSuccess && cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// kern<type or types, VEC> by run-time values
template <typename F> moe_status with_type(int dt, F f)
{
    return dt == MOE_F32 ? f(static_cast<float *>(nullptr)) : f(static_cast<__nv_bfloat16 *>(nullptr));
}
template <typename F> moe_status with_width(bool vec, F f)
{
    return vec ? f(std::true_type()) : f(std::false_type());
}

template <bool WEIGHTED>
moe_status gather_sum(Args a, moe_dtype x_dt, moe_dtype out_dt, cudaStream_t s)
{
    const bool vec = vectors(a.x, a.ldx, a.d) && vectors(a.out, a.ldo, a.d);
    return with_type(x_dt, [&](auto *xt) {
        return with_type(out_dt, [&](auto *ot) {
            return with_width(vec, [&](auto width) {
                using XT = std::remove_pointer_t<decltype(xt)>;
                using OT = std::remove_pointer_t<decltype(ot)>;
                [[maybe_unused]] constexpr bool VEC = decltype(width)::value;
                if constexpr (!WEIGHTED && !std::is_same<XT, OT>::value) return MOE_ERR_INVALID_ARG;   // (never asked for)
                else {
                    dim3 grid;
                    if (!lay_out(a, &grid)) return MOE_ERR_UNSUPPORTED;
                    return launched([&] {
                        return launch_pdl(gather_sum_kernel<XT, OT, VEC, WEIGHTED>, grid, dim3(kThreads), 0, s, a);
                    });
                }
            });
        });
    });
}

}  // namespace rows
}  // namespace moe

using namespace moe;
using namespace moe::rows;

extern "C" {

moe_status moe_dispatch(const void *x, moe_dtype dt, int T, int d, long long ldx, const int32_t *inv, int k, void *out,
                        int rows, long long ldo, moe_stream stream)
{
    bool go;
    const moe_status st = check(T, k, rows, d, inv, &go);
    if (st != MOE_OK) return st;
    if (!matrix_ok(x, dt, ldx, d, T == 0) || !matrix_ok(out, dt, ldo, d, rows == 0 || T == 0)) return MOE_ERR_INVALID_ARG;
    if (!go || rows == 0) return MOE_OK;
    Args a{};
    a.x = x; a.out = out; a.inv = inv; a.ldx = ldx; a.ldo = ldo; a.T = T; a.k = k; a.rows = rows; a.d = d;
    return with_type(dt, [&](auto *xt) {
        return with_width(vectors(x, ldx, d) && vectors(out, ldo, d), [&](auto width) {
            using XT = std::remove_pointer_t<decltype(xt)>;
            constexpr bool VEC = decltype(width)::value;
            dim3 grid;
            if (!lay_out(a, &grid)) return MOE_ERR_UNSUPPORTED;
            return launched([&] {
                return launch_pdl(scatter_rows_kernel<XT, VEC>, grid, dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a);
            });
        });
    });
}

moe_status moe_dispatch_backward(const void *grad, moe_dtype dt, int rows, int d, long long ldg, const int32_t *inv, int T,
                                 int k, void *dx, long long ldx, moe_stream stream)
{
    bool go;
    const moe_status st = check(T, k, rows, d, inv, &go);
    if (st != MOE_OK) return st;
    if (!matrix_ok(grad, dt, ldg, d, rows == 0 || T == 0) || !matrix_ok(dx, dt, ldx, d, T == 0)) return MOE_ERR_INVALID_ARG;
    if (!go) return MOE_OK;
    Args a{};
    a.x = grad; a.out = dx; a.inv = inv; a.ldx = ldg; a.ldo = ldx; a.T = T; a.k = k; a.rows = rows; a.d = d;
    return gather_sum<false>(a, dt, dt, static_cast<cudaStream_t>(stream));
}

moe_status moe_combine(const void *y, moe_dtype y_dt, int rows, int d, long long ldy, const float *topk_w,
                       const int32_t *inv, int T, int k, void *out, moe_dtype out_dt, long long ldo, moe_stream stream)
{
    bool go;
    const moe_status st = check(T, k, rows, d, inv, &go);
    if (st != MOE_OK) return st;
    if (!matrix_ok(y, y_dt, ldy, d, rows == 0 || T == 0) || !matrix_ok(out, out_dt, ldo, d, T == 0)) return MOE_ERR_INVALID_ARG;
    if (!go) return MOE_OK;
    if (!topk_w || !aligned(topk_w, 4)) return MOE_ERR_INVALID_ARG;
    Args a{};
    a.x = y; a.out = out; a.topk_w = topk_w; a.inv = inv; a.ldx = ldy; a.ldo = ldo; a.T = T; a.k = k; a.rows = rows; a.d = d;
    return gather_sum<true>(a, y_dt, out_dt, static_cast<cudaStream_t>(stream));
}

moe_status moe_combine_backward(const void *grad, moe_dtype grad_dt, int T, int d, long long ldg, const void *y,
                                moe_dtype y_dt, int rows, long long ldy, const float *topk_w, const int32_t *inv, int k,
                                void *dy, long long lddy, float *dw, moe_stream stream)
{
    bool go;
    const moe_status st = check(T, k, rows, d, inv, &go);
    if (st != MOE_OK) return st;
    if (!matrix_ok(grad, grad_dt, ldg, d, T == 0) || !matrix_ok(y, y_dt, ldy, d, rows == 0 || T == 0 || !dw))
        return MOE_ERR_INVALID_ARG;
    if ((dy && !matrix_ok(dy, y_dt, lddy, d, true)) || !aligned(dw, 4)) return MOE_ERR_INVALID_ARG;
    if (!go || (!dy && !dw)) return MOE_OK;
    if (!topk_w || !aligned(topk_w, 4)) return MOE_ERR_INVALID_ARG;
    Args a{};
    a.x = y; a.g = grad; a.out = dy; a.dw = dw; a.topk_w = topk_w; a.inv = inv;
    a.ldx = ldy; a.ldg = ldg; a.ldo = lddy; a.T = T; a.k = k; a.rows = rows; a.d = d;
    const bool vec = vectors(grad, ldg, d) && (!dw || vectors(y, ldy, d)) && (!dy || vectors(dy, lddy, d));
    return with_type(y_dt, [&](auto *xt) {
        return with_type(grad_dt, [&](auto *gt) {
            return with_width(vec, [&](auto width) {
                using XT = std::remove_pointer_t<decltype(xt)>;
                using GT = std::remove_pointer_t<decltype(gt)>;
                constexpr bool VEC = decltype(width)::value;
                return launched([&] {
                    cudaStream_t s = static_cast<cudaStream_t>(stream);
                    if (T >= 16 * device_sm_count())
                        return launch_pdl(combine_backward_kernel<XT, GT, VEC, 32>, dim3((unsigned)ceil_div(T, kThreads / 32)),
                                          dim3(kThreads), 0, s, a);
                    return launch_pdl(combine_backward_kernel<XT, GT, VEC, kThreads>, dim3((unsigned)T), dim3(kThreads), 0, s, a);
                });
            });
        });
    });
}

}  // extern "C"
