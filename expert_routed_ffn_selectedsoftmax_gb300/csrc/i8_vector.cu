// i8_vector.cu -- products of a few rows per group on the CUDA cores.
//
// A warp holds four weight rows (PRODUCT: four output channels; GATEUP: two of W_gate
// and the same two of W_up), walks its share of the reduction 512 columns at a time, 16
// bytes a lane, and multiplies each with up to TB tokens' by four-way integer dot products
// (dp4a): sums in 32-bit whole numbers, exact below K = 131072 (where (-128)^2 K is 2^31).
// What bounds it is memory, so what counts is bytes in flight: a long reduction is split over
// the warps of a CTA, until a warp has a step or two (4096 x 4096 of 4 tokens, one warp for
// all of K: 9.1 us).
// Weights are read once for every TB rows of a group.  2048 x 5632 of one token takes 4.4 us:
// all of its 11.5 MB are asked for at once, 1.7 us at the measured copy rate, behind the start.
// Two tokens a group spill 56 bytes at the 64 registers that four CTAs an SM leave; with three CTAs and
// no spill 4096 x 4096 of two tokens takes 7.3 us where it takes 5.5 (2048 x 5632: 4.8 and 4.9).
#include "i8.h"

namespace moe {
namespace i8 {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int NR = 4;                    // weight rows of a warp
constexpr int kStep = 512;               // columns a warp takes at a time

template <int MODE, int TB>
__global__ void __launch_bounds__(kThreads, TB <= 2 ? 4 : TB <= 4 ? 3 : 2)
vector_kernel(const Params p, const int share)   // warps that share a reduction: 1, 2, 4 or 8
{
    pdl_enter();
    constexpr int NW = MODE == GATEUP ? 2 : 1, NC = NR / NW;   // matrices, output channels of a warp
    constexpr int U = TB <= 2 ? 2 : 1;                         // steps in flight
    __shared__ int part[kWarps][NW][NC * TB];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = blockIdx.y;
    const int first = group_bound(p, e), last = group_bound(p, e + 1);
    const int n0 = (blockIdx.x * (kWarps / share) + warp / share) * NC, mine = warp % share;
    const int8_t *w[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int n = min(n0 + i % NC, p.N - 1);   // (channels past the last: not written)
        w[i] = p.w[i / NC] + ((long long)e * p.N + n) * p.K;
    }
    for (int t0 = first; t0 < last; t0 += TB) {    // (the same turns for the whole CTA)
        const int8_t *x[TB];
#pragma unroll
        for (int t = 0; t < TB; ++t) x[t] = p.x_q + source_row(p, min(t0 + t, last - 1)) * p.ldx;
        int acc[NR][TB];
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int t = 0; t < TB; ++t) acc[i][t] = 0;
        const int hop = share * kStep;
#pragma unroll 1
        for (int k0 = mine * kStep + lane * 16; k0 < p.K; k0 += hop * U) {
            int4 a[U][NR];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < NR; ++i)
                    a[u][i] = k0 + hop * u < p.K ? __ldg(reinterpret_cast<const int4 *>(w[i] + k0 + hop * u)) : make_int4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (k0 + hop * u >= p.K) break;
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    const int4 b = __ldg(reinterpret_cast<const int4 *>(x[t] + k0 + hop * u));
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        acc[i][t] = __dp4a(a[u][i].x, b.x, acc[i][t]);
                        acc[i][t] = __dp4a(a[u][i].y, b.y, acc[i][t]);
                        acc[i][t] = __dp4a(a[u][i].z, b.z, acc[i][t]);
                        acc[i][t] = __dp4a(a[u][i].w, b.w, acc[i][t]);
                    }
                }
            }
        }
        // lane c * TB + t has channel c of token t
        int sum[NW];
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                const int s = __reduce_add_sync(0xffffffffu, acc[i][t]);
                if (lane == (i % NC) * TB + t) sum[i / NC] = s;
            }
        const bool has = lane < NC * TB;
        if (share > 1) {
            if (has)
#pragma unroll
                for (int m = 0; m < NW; ++m) part[warp][m][lane] = sum[m];
            __syncthreads();
            if (has && mine == 0)
#pragma unroll
                for (int m = 0; m < NW; ++m)
                    for (int q = 1; q < share; ++q) sum[m] += part[warp + q][m][lane];
            __syncthreads();
        }
        const int t = t0 + lane % TB, n = n0 + lane / TB;
        if (has && mine == 0 && t < last && n < p.N) {
            const float sx = __ldg(p.x_s + source_row(p, t));
            float v[NW];
#pragma unroll
            for (int m = 0; m < NW; ++m) v[m] = (float)sum[m] * sx * __ldg(p.w_s[m] + (long long)e * p.N + n);
            if (MODE == GATEUP) v[0] = p.out_f32 ? swiglu_accurate(v[0], v[NW - 1]) : swiglu_fast(v[0], v[NW - 1]);
            store_out(p, t, n, v[0]);
        }
    }
}

}  // namespace

template <int MODE>
cudaError_t launch_vector(const Params &p, cudaStream_t stream)
{
    constexpr int NC = MODE == GATEUP ? NR / 2 : NR;
    const int experts = p.E < p.rows ? p.E : p.rows, mean = ceil_div(p.rows, experts);
    const int steps = ceil_div(p.K, mean <= 2 ? 2 * kStep : kStep);
    int share = 1;
    while (share < kWarps && share < steps) share *= 2;
    const dim3 grid((unsigned)ceil_div(p.N, NC * (kWarps / share)), (unsigned)p.E), block(kThreads);
    if (mean <= 1) return launch_pdl(vector_kernel<MODE, 1>, grid, block, 0, stream, p, share);
    if (mean <= 2) return launch_pdl(vector_kernel<MODE, 2>, grid, block, 0, stream, p, share);
    if (mean <= 4) return launch_pdl(vector_kernel<MODE, 4>, grid, block, 0, stream, p, share);
    return launch_pdl(vector_kernel<MODE, 8>, grid, block, 0, stream, p, share);
}
template cudaError_t launch_vector<PRODUCT>(const Params &, cudaStream_t);
template cudaError_t launch_vector<GATEUP>(const Params &, cudaStream_t);

}  // namespace i8
}  // namespace moe
