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
// atomic.  A thread holds 8 columns of its token and asks for the k rows' at once.  Sums run
// over the slots in order, in fp32, and are rounded once.
//
// What bounds them is memory.  16384 tokens x 2 of 2048 bf16 columns (us, of the measured copy
// rate): dispatch 30.9, 98 %; its gradient 37.1, 82 %; combine 37.0, 82 %; its gradients 50.6,
// 100 %.  Few tokens are latency: combine of 128 x 2 of 1024 takes 1.5.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace rows {

// Threads of a CTA: dispatch, which only copies, starts too many CTAs of fewer (16384 x 1 x 4096
// 42 us with 256, 66 with 128); sums, whose CTAs end together, are better off with more of
// them (combine of 16384 x 2 x 2048 39.9 and 37.0, of 16384 x 1 x 4096 47.8 and 44.0; 64
// threads as 128 or slower).
constexpr int kCopyThreads = 256, kSumThreads = 128;
constexpr int V = 8;            // columns of a thread's chunk

// V neighbouring columns of a thread, as loaded.
template <typename T> struct Chunk;
template <> struct Chunk<float> {
    uint32_t a[8];
    __device__ __forceinline__ void load(const float *p)
    {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p)), y = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
        a[0] = x.x; a[1] = x.y; a[2] = x.z; a[3] = x.w; a[4] = y.x; a[5] = y.y; a[6] = y.z; a[7] = y.w;
    }
    __device__ __forceinline__ void store(float *p) const
    {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(a[0], a[1], a[2], a[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(a[4], a[5], a[6], a[7]);
    }
    // element i if `in`, else 0 (from i = 0 on, in order)
    __device__ __forceinline__ void load_one(int i, bool in, const float *p)
    {
        a[i] = in ? __ldg(reinterpret_cast<const uint32_t *>(p)) : 0u;
    }
    __device__ __forceinline__ void store_one(int i, float *p) const { *reinterpret_cast<uint32_t *>(p) = a[i]; }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(a[i]); }
    __device__ __forceinline__ void set(const float (&v)[V])
    {
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] = __float_as_uint(v[i]);
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = 0u;
    }
};
template <> struct Chunk<__nv_bfloat16> {
    uint32_t a[4];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p)
    {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p));
        a[0] = x.x; a[1] = x.y; a[2] = x.z; a[3] = x.w;
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = make_uint4(a[0], a[1], a[2], a[3]); }
    __device__ __forceinline__ void load_one(int i, bool in, const __nv_bfloat16 *p)
    {
        const uint32_t v = in ? __ldg(reinterpret_cast<const uint16_t *>(p)) : 0;
        a[i >> 1] = (i & 1) ? a[i >> 1] | (v << 16) : v;
    }
    __device__ __forceinline__ void store_one(int i, __nv_bfloat16 *p) const
    {
        *reinterpret_cast<uint16_t *>(p) = (uint16_t)(a[i >> 1] >> (16 * (i & 1)));
    }
    __device__ __forceinline__ float get(int i) const { return (i & 1) ? bf16hi(a[i >> 1]) : bf16lo(a[i >> 1]); }
    __device__ __forceinline__ void set(const float (&v)[V])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            a[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = 0u;
    }
};

// How a thread's V columns lie.
//   WHOLE    neighbours; rows lie on 16-byte boundaries
//   APART    `step` apart, an element a load: the threads of a row read neighbouring elements.
//            Rows on any boundary, where elements are 4 bytes or little is written.
//   SHIFTED  neighbours that begin on a boundary of the written row, so that stores of
//            2-byte elements are whole too; what is read there comes as the 16-byte pieces
//            around it, shifted into place (only pieces inside the row: at its ends it goes
//            by elements).
// Measured (us, APART / SHIFTED): combine of 4096 x 4 x 2049 in bf16 35.6 / 27.7, in fp32 33.4 /
// 34.5; its gradients in fp32 50.6 / 66.1, of 8192 x 2 x 1001 in bf16 26.2 / 31.3; dispatch's
// gradient of 999 x 3 x 1001 in fp32 5.2 / 5.7, of 4096 x 4 x 2049 33.1 / 33.8, of 8192 x 2 x 1001 in
// bf16 15.4 / 16.2; dispatch there 11.7 / 13.4.  (bf16 goes SHIFTED in all of them, by combine.)
enum Way { WHOLE = 0, APART = 1, SHIFTED = 2 };
template <typename T> __device__ __forceinline__ void load_apart(Chunk<T> &c, const T *p, int step, int left)
{
#pragma unroll
    for (int i = 0; i < V; ++i) c.load_one(i, i * step < left, p + i * step);
}
template <typename T> __device__ __forceinline__ void store_apart(const Chunk<T> &c, T *p, int step, int left)
{
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i * step < left) c.store_one(i, p + i * step);
}
// Columns before the first boundary of a row.
template <typename T> __device__ __forceinline__ int lead_of(const T *row)
{
    return (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T);
}
// Columns col .. col + 7 of a row of d (zeros outside it).
template <typename T> __device__ __forceinline__ void load_any(Chunk<T> &c, const T *row, int col, int d)
{
    constexpr int W = V * (int)sizeof(T) / 4;               // words of a chunk
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + col);
    const int off = (int)(at & 15);
    if (col >= 0 && col + V <= d && off == 0) {
        c.load(row + col);
        return;
    }
    const T *from = reinterpret_cast<const T *>(at - off);
    const int before = off / (int)sizeof(T);
    if (col - before >= 0 && col - before + V + 16 / (int)sizeof(T) <= d) {
        uint32_t w[W + 4];
#pragma unroll
        for (int i = 0; i < W / 4 + 1; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(from) + i);
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
        if (off & 8) {
#pragma unroll
            for (int i = 0; i < W + 2; ++i) w[i] = w[i + 2];
        }
        if (off & 4) {
#pragma unroll
            for (int i = 0; i < W + 1; ++i) w[i] = w[i + 1];
        }
#pragma unroll
        for (int i = 0; i < W; ++i) c.a[i] = (off & 2) ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) c.load_one(i, col + i >= 0 && col + i < d, row + col + i);
}
// ... to a row on one of whose boundaries `col` lies.
template <typename T> __device__ __forceinline__ void store_any(const Chunk<T> &c, T *row, int col, int d)
{
    if (col >= 0 && col + V <= d) {
        c.store(row + col);
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (col + i >= 0 && col + i < d) c.store_one(i, row + col + i);
}

struct Args {
    const void *x;            // dispatch: [T, d]; combine: y [rows, d]
    const void *g;            // combine's backward: [T, d]
    const float *topk_w;      // [T, k], or NULL: weights 1
    const int32_t *inv;       // [T*k]
    void *out;
    float *dw;
    long long ldx, ldg, ldo;  // elements from row to row
    int T, k, rows, d;
    int chunks, col_blocks;   // chunks of a row; CTAs along it
    int each;                 // chunks a thread takes
    int lanes_log2;           // threads of a CTA along a row
    int fill;                 // CTAs ahead of the others that look for rows no slot names
};

// Zeros into the rows that no slot names, for an output whose memory holds nothing yet, by the
// first `fill` CTAs of a grid, beside the others' work.  As many rows as slots all have a slot
// if no slot is without a row: each of these CTAs looks at its share of inv, and goes home
// if all is well there (dispatch of 16384 x 8 x 64: 5.6 us, 5.5 without them, 36 where each
// reads all of inv).  Else those that found a slot without a row share the rows
// among themselves: each marks its own by all of inv (one bit a row in shared memory, as many
// rows at a time as there are bits) and zeroes what stays unmarked.  With a tenth of the slots
// dropped: dispatch of 8192 x 2 x 1024 16 us (8.5), of 16384 x 8 x 64 51 (5.5), combine's
// gradients of 16384 x 2 x 2048 65 (47).
constexpr int kMarkWords = 2048;
template <typename T> __device__ __forceinline__ void zero_row(T *row, int d, int lane)
{
    constexpr int N = 16 / (int)sizeof(T);
    const int lead = min(lead_of(row), d), whole = (d - lead) / N, tail = lead + whole * N;
    Chunk<T> c;
    c.zero();
    if (lane < lead) c.store_one(0, row + lane);
    for (int i = lane; i < whole; i += 32) reinterpret_cast<uint4 *>(row + lead)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tail + lane < d) c.store_one(0, row + tail + lane);
}
// f(number, values) of the fours of slots at(0), at(1), ... up to `hi` of them (U loads of a
// thread in flight).  Ends early once `done` says so.
template <int U, typename AT, typename DONE, typename F>
__device__ __forceinline__ void each_four(const int4 *inv, int fours, int hi, AT at, DONE done, F f)
{
    for (int t = threadIdx.x; t < hi && !done(); t += U * blockDim.x) {
        int4 v[U];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int i = at(t + q * blockDim.x);
            if (i < fours) v[q] = __ldg(inv + i);
        }
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int i = at(t + q * blockDim.x);
            if (i < fours) f(i, v[q]);
        }
    }
}
template <typename T, int U> __device__ __forceinline__ void zero_unnamed(const Args &a)
{
    __shared__ uint32_t named[kMarkWords], found;
    const int lane = threadIdx.x & 31;
    const int n = a.T * a.k;   // (at most kMostMarked)
    const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(a.inv) & 15)) & 15) / 4, n), fours = (n - head) / 4;
    const int4 *inv = reinterpret_cast<const int4 *>(a.inv + head);
    const auto lone = [&](int i) { return __ldg(a.inv + (i < head ? i : i + 4 * fours)); };   // the slots beside the fours
    const int lones = n - 4 * fours;   // (at most 6)
    const auto same = [](int i) { return i; };
    const auto never = [] { return false; };
    uint32_t parts = a.fill, part = blockIdx.x;
    if (n == a.rows) {
        // then there are 1, 2, 4, .. 32 of these CTAs, and a share is every parts-th 64 fours
        const auto without = [&](int r) { return (uint32_t)r >= (uint32_t)a.rows; };
        const auto any = [&](int4 v) { return without(v.x) || without(v.y) || without(v.z) || without(v.w); };
        bool mine = part == 0 && (int)threadIdx.x < lones && without(lone(threadIdx.x));
        each_four<U>(inv, fours, fours / (int)parts + 64, [&](int t) { return ((t >> 6) * (int)parts + (int)part) * 64 + (t & 63); }, never,
                     [&](int, int4 v) { mine |= any(v); });
        if (threadIdx.x == 0) found = 0u;
        if (!__syncthreads_or(mine)) return;
        const uint32_t all = parts == 32 ? 0xffffffffu : (1u << parts) - 1u;
        if ((int)threadIdx.x < lones && without(lone(threadIdx.x))) atomicOr(&found, 1u);
        each_four<U>(inv, fours, fours, same, [&] { return *static_cast<volatile uint32_t *>(&found) == all; },
                     [&](int i, int4 v) { if (any(v)) atomicOr(&found, 1u << ((i >> 6) & (parts - 1))); });
        __syncthreads();
        part = __popc(found & ((1u << part) - 1u));
        parts = __popc(found);
    }
    uint32_t first = (uint32_t)((uint64_t)a.rows * part / parts);
    uint32_t rows = (uint32_t)((uint64_t)a.rows * (part + 1) / parts) - first;
    while (rows > 0) {
        const uint32_t count = min(rows, kMarkWords * 32u);
        for (int i = threadIdx.x; i < kMarkWords; i += blockDim.x) named[i] = 0u;
        __syncthreads();
        const auto mark = [&](int r) {
            const uint32_t at = (uint32_t)r - first;   // (negative indexes are beyond any count)
            if (at < count) atomicOr(&named[at >> 5], 1u << (at & 31));
        };
        each_four<U>(inv, fours, fours, same, never, [&](int, int4 v) { mark(v.x); mark(v.y); mark(v.z); mark(v.w); });
        if ((int)threadIdx.x < lones) mark(lone(threadIdx.x));
        __syncthreads();
        for (uint32_t w = threadIdx.x >> 5; w * 32 < count; w += blockDim.x >> 5) {
            uint32_t left = ~named[w];
            if (count - w * 32 < 32) left &= (1u << (count - w * 32)) - 1u;
            for (; left; left &= left - 1u)
                zero_row(static_cast<T *>(a.out) + (long long)(first + w * 32 + (__ffs(left) - 1)) * a.ldo, a.d, lane);
        }
        __syncthreads();
        first += count;
        rows -= count;
    }
}

// This thread's token and chunk; a CTA holds blockDim.x >> lanes_log2 tokens, and a row's
// chunks are spread over col_blocks CTAs.
__device__ __forceinline__ bool place(const Args &a, long long &t, int &chunk)
{
    const int lanes = 1 << a.lanes_log2;
    const uint32_t block = blockIdx.x - a.fill;
    const long long tb = block / a.col_blocks;
    t = tb * (blockDim.x >> a.lanes_log2) + (threadIdx.x >> a.lanes_log2);
    chunk = (int)(block - tb * a.col_blocks) * (lanes * a.each) + (threadIdx.x & (lanes - 1));
    return t < a.T && chunk < a.chunks;
}
// The first column of chunk c (SHIFTED: chunk 0 is what stands before the first boundary).
template <int WAY, typename T> __device__ __forceinline__ int column(int c, int lanes, const T *written)
{
    const int lane = c & (lanes - 1);   // (lanes is a power of two)
    return WAY == WHOLE ? c * V : WAY == APART ? (c - lane) * V + lane : lead_of(written) + (c - 1) * V;
}
template <int WAY, typename T> __device__ __forceinline__ void load(Chunk<T> &c, const T *row, int col, int lanes, int d)
{
    if (WAY == WHOLE) c.load(row + col);
    else if (WAY == APART) load_apart(c, row + col, lanes, d - col);
    else load_any(c, row, col, d);
}
template <int WAY, typename T> __device__ __forceinline__ void store(const Chunk<T> &c, T *row, int col, int lanes, int d)
{
    if (WAY == WHOLE) c.store(row + col);
    else if (WAY == APART) store_apart(c, row + col, lanes, d - col);
    else store_any(c, row, col, d);
}

template <typename XT, int WAY>
// (CTAs an SM: with 34 registers a thread, seven, 16384 x 1 x 4096 takes 47.3 us, with 32 42.3; element
// loads want registers: 6545 x 1 x 124 in fp32 3.4 us with 32, 3.0 with 36)
__global__ void __launch_bounds__(kCopyThreads, WAY == APART ? 6 : 8)
scatter_rows_kernel(const Args a)
{
    pdl_enter();
    if (__builtin_expect(blockIdx.x < (uint32_t)a.fill, 0)) {
        zero_unnamed<XT, 2>(a);
        return;
    }
    long long t;
    int chunk;
    if (!place(a, t, chunk)) return;
    const int lanes = 1 << a.lanes_log2;
    const XT *x = static_cast<const XT *>(a.x) + t * a.ldx;
    const int32_t *inv = a.inv + t * a.k;
    Chunk<XT> c;
    if (WAY != SHIFTED) load<WAY>(c, x, column<WAY>(chunk, lanes, x), lanes, a.d);
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {
        const int r = __ldg(inv + j);
        if (r < 0 || r >= a.rows) continue;
        XT *out = static_cast<XT *>(a.out) + r * a.ldo;
        const int col = column<WAY>(chunk, lanes, out);
        if (WAY == SHIFTED) load<WAY>(c, x, col, lanes, a.d);
        store<WAY>(c, out, col, lanes, a.d);
    }
}

// WEIGHTED: combine; else dispatch's backward pass.  A thread takes EACH chunks, lanes
// apart, and asks for U rows of them at once.
template <typename XT, typename OT, int WAY, bool WEIGHTED, int EACH, int U>
__global__ void __launch_bounds__(kSumThreads)
gather_sum_kernel(const Args a)
{
    pdl_enter();
    long long t;
    int chunk;
    if (!place(a, t, chunk)) return;
    const int lanes = 1 << a.lanes_log2;
    OT *out = static_cast<OT *>(a.out) + t * a.ldo;
    const XT *x = static_cast<const XT *>(a.x);
    const int32_t *inv = a.inv + t * a.k;
    const float *w = a.topk_w + t * a.k;
    float sum[EACH][V];
#pragma unroll
    for (int e = 0; e < EACH; ++e)
#pragma unroll
        for (int i = 0; i < V; ++i) sum[e][i] = 0.f;
    for (int j0 = 0; j0 < a.k; j0 += U) {
        Chunk<XT> c[EACH][U];
        float f[U];
        bool in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = j0 + u < a.k ? __ldg(inv + j0 + u) : -1;
            in[u] = r >= 0 && r < a.rows;
            f[u] = 1.f;
            if (in[u]) {
#pragma unroll
                for (int e = 0; e < EACH; ++e) {
                    const int at = chunk + e * lanes;
                    if (at < a.chunks) load<WAY>(c[e][u], x + r * a.ldx, column<WAY>(at, lanes, out), lanes, a.d);
                }
                if (WEIGHTED) f[u] = __ldg(w + j0 + u);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!in[u]) continue;   // (a slot without a row adds nothing, whatever its weight)
#pragma unroll
            for (int e = 0; e < EACH; ++e)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    sum[e][i] = WEIGHTED ? fmaf(f[u], c[e][u].get(i), sum[e][i]) : sum[e][i] + c[e][u].get(i);
        }
    }
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        const int at = chunk + e * lanes;
        if (at >= a.chunks) break;
        Chunk<OT> o;
        o.set(sum[e]);
        store<WAY>(o, out, column<WAY>(at, lanes, out), lanes, a.d);
    }
}

// Combine's backward pass: a token to a group of `G` threads (a warp, or a CTA),
// which walk its chunks; each thread sums its part of every slot's product, and the
// parts meet in a fixed order (shuffles, then the warps in order).
constexpr int backward_threads(int G) { return G == 32 ? 128 : G; }
template <typename XT, typename GT, int WAY, int G>
__global__ void __launch_bounds__(backward_threads(G))
combine_backward_kernel(const Args a)
{
    pdl_enter();
    constexpr int N = backward_threads(G);
    if (__builtin_expect(blockIdx.x < (uint32_t)a.fill, 0)) {
        zero_unnamed<XT, 8>(a);
        return;
    }
    __shared__ float part[N / 32][kMaxTopK];
    const int lane = threadIdx.x & (G - 1);
    const long long t = (long long)(blockIdx.x - a.fill) * (N / G) + threadIdx.x / G;
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
        // a row's share of a chunk: its part of the dot product, and its gradient
        auto finish = [&](int j, const Chunk<GT> &c, const Chunk<XT> &v, int col) {
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dot[j] = fmaf(c.get(i), v.get(i), dot[j]);
                o[i] = w[j] * c.get(i);
            }
            if (dy) {
                Chunk<XT> s;
                s.set(o);
                store<WAY>(s, dy + r[j] * a.ldo, col, G, a.d);
            }
        };
        if constexpr (WAY == SHIFTED) {
            for (int chunk = lane; chunk < a.chunks; chunk += G) {
                // (two rows at a time: their loads stand ahead of the stores)
#pragma unroll
                for (int j0 = 0; j0 < kMaxTopK; j0 += 2) {
                    if (j0 >= a.k) break;
                    Chunk<XT> v[2];
                    Chunk<GT> c[2];   // the gradient at each row's own columns
                    int col[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int j = j0 + u;
                        if (r[j] < 0) continue;
                        // (without dy nothing is written: y's rows decide)
                        col[u] = column<WAY>(chunk, G, dy ? dy + r[j] * a.ldo : y + r[j] * a.ldx);
                        v[u].zero();
                        if (a.dw) load_any(v[u], y + r[j] * a.ldx, col[u], a.d);
                        load_any(c[u], g, col[u], a.d);
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        if (r[j0 + u] >= 0) finish(j0 + u, c[u], v[u], col[u]);
                }
            }
        } else {
            constexpr int C = WAY == WHOLE ? 2 : 1;   // chunks in flight
            for (int c0 = lane; c0 < a.chunks; c0 += C * G) {
                Chunk<GT> c[C];
#pragma unroll
                for (int q = 0; q < C; ++q)
                    if (c0 + q * G < a.chunks) load<WAY>(c[q], g, column<WAY>(c0 + q * G, G, g), G, a.d);
#pragma unroll
                for (int j0 = 0; j0 < kMaxTopK; j0 += 2) {
                    if (j0 >= a.k) break;
                    Chunk<XT> v[C][2];
#pragma unroll
                    for (int q = 0; q < C; ++q)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            v[q][u].zero();
                            if (r[j0 + u] >= 0 && a.dw && c0 + q * G < a.chunks)
                                load<WAY>(v[q][u], y + r[j0 + u] * a.ldx, column<WAY>(c0 + q * G, G, y), G, a.d);
                        }
#pragma unroll
                    for (int q = 0; q < C; ++q)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            if (r[j0 + u] >= 0 && c0 + q * G < a.chunks) finish(j0 + u, c[q], v[q][u], column<WAY>(c0 + q * G, G, y));
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
    if (k > kMaxTopK || d > kMostColumns) return MOE_ERR_UNSUPPORTED;
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

// Chunks of a row that have columns.  SHIFTED: one more, for what stands before its first
// boundary; APART: `lanes` of them hold lanes * V columns together, and the last lanes' are
// the shorter ones.
int chunks_of(int d, int way, int lanes)
{
    if (way == APART) return d / (lanes * V) * lanes + (d % (lanes * V) < lanes ? d % (lanes * V) : lanes);
    return ceil_div(d, V) + (way == SHIFTED);
}
// grid of a kernel whose threads, `cta` to a CTA, take `each` chunks
bool lay_out(Args &a, int way, int each, int cta, dim3 *grid)
{
    const int threads = ceil_div(chunks_of(a.d, way == APART ? WHOLE : way, 1), each);
    a.lanes_log2 = 5;
    while ((1 << a.lanes_log2) < cta && (1 << a.lanes_log2) < threads) ++a.lanes_log2;
    a.chunks = chunks_of(a.d, way, 1 << a.lanes_log2);
    a.each = each;
    a.col_blocks = ceil_div(a.chunks, each << a.lanes_log2);
    const int per = cta >> a.lanes_log2;
    const long long ctas = ((long long)a.T + per - 1) / per * a.col_blocks + a.fill;
    *grid = dim3((unsigned)ctas);
    return ctas <= 0x7fffffffLL;
}

// The CTAs that look for rows no slot names: 1, 2, 4, .. 32, one for 1024 rows, more for
// rows that no slot can name.  They read inv once for every kMarkWords * 32 rows, so beyond
// kMostMarked slots the rows are zeroed as a whole ahead (`all`: the grid is these CTAs alone,
// and no slot names a row).
constexpr long long kMostMarked = 1 << 21;
void plan_fill(Args &a, bool all)
{
    if (all) a.T = 0;
    const long long rows = a.rows, n = (long long)a.T * a.k;
    a.fill = 1;
    while (a.fill < 32 && a.fill * 1024LL < rows) a.fill *= 2;
    if (rows <= n) return;
    const long long more = (rows - n) / 64, most = 4LL * device_sm_count();
    a.fill += (int)(more < most ? more : most);
}

template <typename F> moe_status launched(F launch)
{
    return launch() == cudaSuccess && cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// A launch that writes grouped rows, `filled` or not: with its fill plan, or behind one that
// zeroes every row.
template <typename F> moe_status with_fill(const Args &a, bool filled, F launch)
{
    Args b = a;
    if (!filled) return launch(b);
    const bool all = a.T == 0 || (long long)a.T * a.k > kMostMarked;
    plan_fill(b, all);
    const moe_status st = launch(b);
    return all && a.T > 0 && st == MOE_OK ? launch(a) : st;
}

// a kernel's types by run-time values
template <typename F> moe_status with_type(int dt, F f)
{
    return dt == MOE_F32 ? f(static_cast<float *>(nullptr)) : f(static_cast<__nv_bfloat16 *>(nullptr));
}
template <int WAY> using WayOf = std::integral_constant<int, WAY>;

template <typename XT, typename OT, int WAY, bool WEIGHTED>
moe_status launch_gather_sum(Args a, cudaStream_t s)
{
    // Many tokens: about 64 bytes in flight a thread (combine of 16384 x 2 x 2048 in bf16: one
    // chunk a thread 38.2 us, two 37.0); few: a chunk a thread and its rows at once, as that is
    // latency, with registers for no more of them than there are (4096 x 2 x 1024: two at once
    // 6.6, four 7.2; 16384 x 4 x 1024 30.1 and 28.5).
    const bool many = (long long)a.T * (a.d / V) >= 4096LL * device_sm_count();
    constexpr int kTwice = sizeof(XT) == 4 ? 1 : 2;   // (fp32 chunks are twice as long)
    const auto go = [&](auto kern, int each) {
        dim3 grid;
        if (!lay_out(a, WAY, each, kSumThreads, &grid)) return MOE_ERR_UNSUPPORTED;
        return launched([&] { return launch_pdl(kern, grid, dim3(kSumThreads), 0, s, a); });
    };
    if constexpr (WAY == WHOLE) {
        if (many && a.k == 1) return go(gather_sum_kernel<XT, OT, WAY, WEIGHTED, 2 * kTwice, 1>, 2 * kTwice);
        if (many && a.k <= 3) return go(gather_sum_kernel<XT, OT, WAY, WEIGHTED, kTwice, 2>, kTwice);
        if (a.k > 2) return go(gather_sum_kernel<XT, OT, WAY, WEIGHTED, 1, 4>, 1);
    }
    return go(gather_sum_kernel<XT, OT, WAY, WEIGHTED, 1, 2>, 1);
}

template <bool WEIGHTED>
moe_status gather_sum(const Args &a, moe_dtype x_dt, moe_dtype out_dt, cudaStream_t s)
{
    const bool whole = vectors(a.x, a.ldx, a.d) && vectors(a.out, a.ldo, a.d);
    return with_type(x_dt, [&](auto *xt) {
        return with_type(out_dt, [&](auto *ot) {
            using XT = std::remove_pointer_t<decltype(xt)>;
            using OT = std::remove_pointer_t<decltype(ot)>;
            if constexpr (!WEIGHTED && !std::is_same<XT, OT>::value) return MOE_ERR_INVALID_ARG;   // (never asked for)
            else return whole ? launch_gather_sum<XT, OT, WHOLE, WEIGHTED>(a, s) : launch_gather_sum<XT, OT, sizeof(XT) == 4 ? APART : SHIFTED, WEIGHTED>(a, s);
        });
    });
}

// `filled`: rows of the output that no slot names become zeros.
moe_status dispatch(const void *x, moe_dtype dt, int T, int d, long long ldx, const int32_t *inv, int k, void *out, int rows,
                    long long ldo, bool filled, cudaStream_t stream)
{
    bool go;
    const moe_status st = check(T, k, rows, d, inv, &go);
    if (st != MOE_OK) return st;
    if (!matrix_ok(x, dt, ldx, d, T == 0) || !matrix_ok(out, dt, ldo, d, rows == 0 || (T == 0 && !filled))) return MOE_ERR_INVALID_ARG;
    if (rows == 0 || (!go && !filled)) return MOE_OK;
    Args a{};
    a.x = x; a.out = out; a.inv = inv; a.ldx = ldx; a.ldo = ldo; a.T = T; a.k = k; a.rows = rows; a.d = d;
    return with_type(dt, [&](auto *xt) {
        using XT = std::remove_pointer_t<decltype(xt)>;
        constexpr int kOff = sizeof(XT) == 4 ? APART : SHIFTED;
        const auto go = [&](auto kern, int way) {
            return with_fill(a, filled, [&](Args b) {
                dim3 grid;
                if (!lay_out(b, way, 1, kCopyThreads, &grid)) return MOE_ERR_UNSUPPORTED;
                return launched([&] { return launch_pdl(kern, grid, dim3(kCopyThreads), 0, stream, b); });
            });
        };
        if (vectors(x, ldx, d) && vectors(out, ldo, d)) return go(scatter_rows_kernel<XT, WHOLE>, WHOLE);
        return go(scatter_rows_kernel<XT, kOff>, kOff);
    });
}

moe_status combine_backward(const void *grad, moe_dtype grad_dt, int T, int d, long long ldg, const void *y, moe_dtype y_dt,
                            int rows, long long ldy, const float *topk_w, const int32_t *inv, int k, void *dy, long long lddy,
                            float *dw, bool filled, cudaStream_t stream)
{
    bool go;
    const moe_status st = check(T, k, rows, d, inv, &go);
    if (st != MOE_OK) return st;
    if (!matrix_ok(grad, grad_dt, ldg, d, T == 0) || !matrix_ok(y, y_dt, ldy, d, rows == 0 || T == 0 || !dw))
        return MOE_ERR_INVALID_ARG;
    if ((dy && !matrix_ok(dy, y_dt, lddy, d, true)) || !aligned(dw, 4)) return MOE_ERR_INVALID_ARG;
    filled = filled && dy && rows > 0;
    if ((!go && !filled) || (!dy && !dw)) return MOE_OK;
    if (go && (!topk_w || !aligned(topk_w, 4))) return MOE_ERR_INVALID_ARG;
    Args a{};
    a.x = y; a.g = grad; a.out = dy; a.dw = dw; a.topk_w = topk_w; a.inv = inv;
    a.ldx = ldy; a.ldg = ldg; a.ldo = lddy; a.T = T; a.k = k; a.rows = rows; a.d = d;
    const bool whole = vectors(grad, ldg, d) && (!dw || vectors(y, ldy, d)) && (!dy || vectors(dy, lddy, d));
    return with_type(y_dt, [&](auto *xt) {
        return with_type(grad_dt, [&](auto *gt) {
            using XT = std::remove_pointer_t<decltype(xt)>;
            using GT = std::remove_pointer_t<decltype(gt)>;
            constexpr int kOff = sizeof(XT) == 4 ? APART : SHIFTED;
            const auto go = [&](auto way) {
                constexpr int WAY = decltype(way)::value;
                // Threads of a token.  Many tokens: a warp, or two where it has more than two
                // chunks a lane; few: as many as their chunks keep in use.  us, 32 / 64 / 128 / 512:
                // 16384 x 2 x 128 10.8 / 18.8 / 29.5, x 2048 51.3 / 50.7 / 53.1; 1945 x 7 x 278
                // 18.3 / 19.2 / 21.1; 999 x 3 x 1000 6.8 / 5.3 / 5.3 / 13.4; 3000 x 8 x 8192
                // 135 / 137 / 130 / 131; 300 x 4 x 4096 18.4 / 11.0 / 7.6 / 6.4; 64 x 2 x 2048 3.6 / 2.6 /
                // 2.0 / 2.1; 16 x 2 x 8192 10.5 / 5.8 / 3.7 / 2.5.
                const int sms = device_sm_count(), chunks = ceil_div(d, V);
                const auto launch = [&](auto group) {
                    constexpr int G = decltype(group)::value, N = backward_threads(G);
                    return with_fill(a, filled, [&](Args b) {
                        b.chunks = chunks_of(d, WAY, G);
                        const long long ctas = (long long)ceil_div(b.T, N / G) + b.fill;
                        return launched([&] {
                            return launch_pdl(combine_backward_kernel<XT, GT, WAY, G>, dim3((unsigned)ctas), dim3(N), 0, stream, b);
                        });
                    });
                };
                if (T >= 10 * sms && chunks <= 64) return launch(std::integral_constant<int, 32>());
                if (chunks <= 64 || (T >= 10 * sms && chunks < 1024)) return launch(std::integral_constant<int, 64>());
                if (T <= 2 * sms && chunks > 256) return launch(std::integral_constant<int, 512>());
                return launch(std::integral_constant<int, 128>());
            };
            return whole ? go(WayOf<WHOLE>()) : go(WayOf<kOff>());
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
    return dispatch(x, dt, T, d, ldx, inv, k, out, rows, ldo, false, static_cast<cudaStream_t>(stream));
}

moe_status moe_dispatch_filled(const void *x, moe_dtype dt, int T, int d, long long ldx, const int32_t *inv, int k, void *out,
                               int rows, long long ldo, moe_stream stream)
{
    return dispatch(x, dt, T, d, ldx, inv, k, out, rows, ldo, true, static_cast<cudaStream_t>(stream));
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
    return combine_backward(grad, grad_dt, T, d, ldg, y, y_dt, rows, ldy, topk_w, inv, k, dy, lddy, dw, false,
                            static_cast<cudaStream_t>(stream));
}

moe_status moe_combine_backward_filled(const void *grad, moe_dtype grad_dt, int T, int d, long long ldg, const void *y,
                                       moe_dtype y_dt, int rows, long long ldy, const float *topk_w, const int32_t *inv,
                                       int k, void *dy, long long lddy, float *dw, moe_stream stream)
{
    return combine_backward(grad, grad_dt, T, d, ldg, y, y_dt, rows, ldy, topk_w, inv, k, dy, lddy, dw, true,
                            static_cast<cudaStream_t>(stream));
}

}  // extern "C"
