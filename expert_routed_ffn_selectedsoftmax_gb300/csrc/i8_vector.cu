// i8_vector.cu -- products of a few rows per group on the CUDA cores.
//
// A warp holds four weight rows (PRODUCT: four output channels; GATEUP: two of W_gate
// and the same two of W_up), walks the reduction 512 columns at a time, 16 bytes a
// lane, and multiplies each with up to TB tokens' by four-way integer dot products
// (dp4a): sums in 32-bit whole numbers, exact up to K = 131072.  The lanes' sums meet
// at the end of the walk.  Weights are read once for every TB rows of a group.
#include "i8.h"

namespace moe {
namespace i8 {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int NR = 4;                    // weight rows of a warp

template <int MODE, int TB>
__global__ void __launch_bounds__(kThreads)
vector_kernel(const Params p)
{
    pdl_enter();
    constexpr int NW = MODE == GATEUP ? 2 : 1, NC = NR / NW;   // matrices, output channels of a warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = blockIdx.y;
    const int first = group_bound(p, e), last = group_bound(p, e + 1);
    const int n0 = (blockIdx.x * kWarps + warp) * NC;
    if (n0 >= p.N) return;
    const int8_t *w[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int n = min(n0 + i % NC, p.N - 1);   // (channels past the last: not written)
        w[i] = p.w[i / NC] + ((long long)e * p.N + n) * p.K;
    }
    for (int t0 = first; t0 < last; t0 += TB) {
        const int8_t *x[TB];
#pragma unroll
        for (int t = 0; t < TB; ++t) x[t] = p.x_q + source_row(p, min(t0 + t, last - 1)) * p.ldx;
        int acc[NR][TB];
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int t = 0; t < TB; ++t) acc[i][t] = 0;
        constexpr int U = TB <= 2 ? 2 : 1;   // steps of 512 columns in flight
        for (int k0 = lane * 16; k0 < p.K; k0 += 512 * U) {
            int4 a[U][NR];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < NR; ++i)
                    a[u][i] = k0 + 512 * u < p.K ? __ldg(reinterpret_cast<const int4 *>(w[i] + k0 + 512 * u)) : make_int4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (k0 + 512 * u >= p.K) break;
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    const int4 b = __ldg(reinterpret_cast<const int4 *>(x[t] + k0 + 512 * u));
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
        // lane c * TB + t finishes channel c of token t
        int mine[NW];
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                const int s = __reduce_add_sync(0xffffffffu, acc[i][t]);
                if (lane == (i % NC) * TB + t) mine[i / NC] = s;
            }
        const int c = lane / TB, t = t0 + lane % TB, n = n0 + c;
        if (c < NC && t < last && n < p.N) {
            const float sx = __ldg(p.x_s + source_row(p, t));
            float v[NW];
#pragma unroll
            for (int m = 0; m < NW; ++m) v[m] = (float)mine[m] * sx * __ldg(p.w_s[m] + (long long)e * p.N + n);
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
    const dim3 grid((unsigned)ceil_div(p.N, NC * kWarps), (unsigned)p.E), block(kThreads);
    const int experts = p.E < p.rows ? p.E : p.rows;
    const int mean = ceil_div(p.rows, experts);
    if (mean <= 1) return launch_pdl(vector_kernel<MODE, 1>, grid, block, 0, stream, p);
    if (mean <= 2) return launch_pdl(vector_kernel<MODE, 2>, grid, block, 0, stream, p);
    if (mean <= 4) return launch_pdl(vector_kernel<MODE, 4>, grid, block, 0, stream, p);
    return launch_pdl(vector_kernel<MODE, 8>, grid, block, 0, stream, p);
}
template cudaError_t launch_vector<PRODUCT>(const Params &, cudaStream_t);
template cudaError_t launch_vector<GATEUP>(const Params &, cudaStream_t);

}  // namespace i8
}  // namespace moe
