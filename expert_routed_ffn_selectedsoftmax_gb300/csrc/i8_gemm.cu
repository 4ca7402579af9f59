// i8_gemm.cu -- products of int8 matrices with a scale for each token and each output
// channel: the calls, and which kernel takes them.
//
//   y[r,n] = (sum_i cx[r,i] cw[n,i]) sx[r] sw[n]
#include "i8.h"

namespace moe {
namespace i8 {

constexpr int kFewRows = 32;   // up to here no call takes the tiled kernel, and none needs a workspace

// The CUDA-core kernel: one or two rows, or up to 32 with at most 8 a group and 6e7
// products.  It starts without barriers, tensor maps and TMEM, but a row costs it a pass of
// dot products where the tensor cores take 32 at once.  us a call (here / few rows):
// 2048 x 5632 of 1 token 4.4 / 6.9, 4: 6.6 / 7.2, 8: 9.1 / 7.5; 1024 x 1024 of 8 2.5 / 3.7;
// 8192 x 8192 of 1 14.5 / 18.3, 4: 19.0 / 18.7; 8 rows over 16 experts of 2816 x 2048
// 11.3 / 13.4, 64 over 64 of 512 x 1024 11.5 / 8.3; gate/up of 16 tokens x 2 over 64
// experts of 1024 x 512 8.3 / 9.7, of 64 rows 16.4 / 10.8.
template <int MODE> bool vector_fits(const Params &p, long long experts)
{
    if (p.K >= 131072) return false;   // (its sums are 32-bit whole numbers)
    if (p.rows <= 2) return true;
    return p.rows <= kFewRows && p.rows <= 8 * experts &&
           (double)p.rows * p.N * p.K * (MODE == GATEUP ? 2 : 1) <= 6e7;
}

// Few rows or tiled, by what each is expected to take (us).  The few-rows kernel takes
// blocks of 128 columns in 0.39 us where every tile has an SM and 0.62 where two share one,
// and a tile's end in 0.6 (SwiGLU's 1.0); the tiled kernel takes 0.335 and a tile's end 0.8, on
// a quarter of the tiles, but it starts later (its rows are widened first).  Where a reduction is split, a CTA has its
// share of the blocks, and its cluster's meeting.  A tile more than the SMs have places for is
// a round more; the groups' sizes are known on the device only, so there their last tiles are
// taken as half full, and a tenth of a round more as none.
// Measured (few rows / tiled): 4096 x 4096 of 64 rows 13.6 / 12.6, 128: 16.0 / 14.1, 300:
// 33.0 / 19.1; 2048 x 5632 of 128 13.6 / 12.7; 1024 x 1024 of 1024 8.8 / 9.9, 2048: 14.4 / 10.9;
// 2048 x 2048 of 128 10.0 / 12.1; 8192 x 1024 of 256 18.6 / 15.7, 1024: 42.0 / 25.3; 64
// experts of 2048 x 1024, rows per expert 16: 28.0 / 33.3, 32: 35.4 / 37.3, 47: 44.6 / 38.9;
// 16 of 2816 x 2048, 24: 25.6 / 26.6, 40: 32.3 / 27.8; gate/up, 64 of 1024 x 512, 16: 18.0 /
// 22.0, 64: 33.6 / 28.0; one of 2048 x 5632, 100 rows: 26.7 / 14.5; two of 160 x 2805, 742 rows
// each: 27.4 / 17.0.
template <int MODE> bool few_rows_fit(const Params &p, int experts)
{
    if (p.rows <= kFewRows) return true;
    const int sms = device_sm_count(), blocks = ceil_div(p.K, kBlock), columns = ceil_div(p.N, channels_of_tile(MODE));
    const auto rounds = [&](int tokens, int places) {
        if (experts == 1) return ceil((double)ceil_div(p.rows, tokens) * columns / places);
        const double each = (double)p.rows / tokens + experts * 0.5;
        const double r = ceil((each > experts ? each : experts) * columns / places - 0.1);
        return r > 1 ? r : 1;
    };
    const int split = split_of(most_tiles(p.rows, experts, 32) * columns, blocks, sms);
    const double few = split > 1 ? 6.5 + 0.39 * ceil_div(blocks, split)
                     : rounds(32, sms) <= 1 ? 3.5 + 0.39 * blocks
                                            : 3.5 + (0.62 * blocks + (MODE == GATEUP ? 1.0 : 0.6)) * rounds(32, 2 * sms);
    const int tiled_split = split_of_tiled<MODE>(most_tiles(p.rows, experts, 128) * columns, blocks);
    const double tiled = 6.3 + (double)p.rows * p.K * 3.4e-7 +
                         (tiled_split > 1 ? 5 + 0.335 * ceil_div(blocks, tiled_split) : rounds(128, sms) * (0.335 * blocks + 0.8));
    return few <= tiled;
}

template <int MODE> cudaError_t launch_product(const Params &p, void *workspace, cudaStream_t stream)
{
    const int experts = p.E < p.rows ? p.E : p.rows;
    if (p.expire_ns == 0 && vector_fits<MODE>(p, experts)) return launch_vector<MODE>(p, stream);   // (it has no waits)
    if (few_rows_fit<MODE>(p, experts)) return launch_few<MODE>(p, stream);
    return launch_tiled<MODE>(p, workspace, stream);
}

bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The checks the products share; MOE_OK with *go = false for an empty call.
moe_status product_args(const Params &p, moe_dtype out_dt, const void *workspace, size_t ws_bytes, bool *go)
{
    *go = false;
    if (p.x_rows < 0 || p.rows < 0 || p.K <= 0 || p.K % 16 || p.N <= 0 || p.E <= 0) return MOE_ERR_INVALID_ARG;
    if (p.ldx < p.K || p.ldx % 16 || p.ldo < p.N) return MOE_ERR_INVALID_ARG;
    if (out_dt != MOE_F32 && out_dt != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (p.E > kMaxExperts || p.K > kMostColumns || p.N > kMostColumns) return MOE_ERR_UNSUPPORTED;
    if (p.E > 1 && !p.offsets && p.rows > 0) return MOE_ERR_INVALID_ARG;
    if (p.rows == 0) return MOE_OK;
    if (!p.perm_tok && p.rows > p.x_rows) return MOE_ERR_INVALID_ARG;
    if (p.x_rows == 0) return MOE_ERR_INVALID_ARG;
    if (p.rows > INT32_MAX / 2 || p.x_rows > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
    if (!p.x_q || !p.x_s || !p.w[0] || !p.w_s[0] || !p.w[1] || !p.w_s[1] || !p.out) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(p.x_q, 16) || !aligned_to(p.x_s, 4) || !aligned_to(p.offsets, 4) || !aligned_to(p.perm_tok, 4) ||
        !aligned_to(p.status, 4) || !aligned_to(p.out, out_dt == MOE_F32 ? 4 : 2))
        return MOE_ERR_INVALID_ARG;
    for (int m = 0; m < 2; ++m)
        if (!aligned_to(p.w[m], 16) || !aligned_to(p.w_s[m], 4)) return MOE_ERR_INVALID_ARG;
    const size_t need = moe_i8_workspace_size(p.rows, p.K);
    if (need && (!workspace || !aligned_to(workspace, 256))) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE;
    *go = true;
    return MOE_OK;
}

template <int MODE>
moe_status product(const void *x_q, const float *x_s, int x_rows, int K, long long ldx, const void *w0, const float *s0,
                   const void *w1, const float *s1, int E, int N, const int32_t *offsets, const int32_t *perm_tok, int rows,
                   void *out, moe_dtype out_dt, long long ldo, void *workspace, size_t ws_bytes, uint32_t *status,
                   int expire_role, uint32_t expire_ns, moe_stream stream)
{
    Params p{};
    p.x_q = static_cast<const int8_t *>(x_q); p.x_s = x_s;
    p.w[0] = static_cast<const int8_t *>(w0); p.w[1] = static_cast<const int8_t *>(w1);
    p.w_s[0] = s0; p.w_s[1] = s1;
    p.offsets = offsets; p.perm_tok = perm_tok;
    p.ldx = ldx; p.ldo = ldo;
    p.E = E; p.rows = rows; p.x_rows = x_rows; p.K = K; p.N = N;
    p.out = out; p.out_f32 = out_dt == MOE_F32;
    const int v = out_dt == MOE_F32 ? 4 : 8;
    p.out_vec = N % v == 0 && ldo % v == 0 && aligned_to(out, 16);
    p.status = status; p.expire_ns = expire_ns; p.expire_role = expire_role;
    bool go;
    const moe_status st = product_args(p, out_dt, workspace, ws_bytes, &go);
    if (st != MOE_OK || !go) return st;
    const cudaError_t e = launch_product<MODE>(p, workspace, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace i8
}  // namespace moe

using namespace moe;
using namespace moe::i8;

namespace {

bool hook_ok(int role, uint32_t wait_ns) { return role >= LOADS && role <= SUMS && wait_ns > 0 && wait_ns <= 100000000u; }

}  // namespace

extern "C" {

size_t moe_i8_workspace_size(int rows, int K)
{
    if (rows <= kFewRows || K <= 0 || K % 16) return 0;
    return tiled_workspace(rows, K);
}

moe_status moe_grouped_gemm_i8(const void *x_q, const float *x_s, int x_rows, int K, long long ldx, const void *w_q,
                               const float *w_s, int E, int N, const int32_t *offsets, const int32_t *perm_tok, int rows,
                               void *out, moe_dtype out_dt, long long ldo, void *workspace, size_t ws_bytes,
                               uint32_t *status, moe_stream stream)
{
    return product<PRODUCT>(x_q, x_s, x_rows, K, ldx, w_q, w_s, w_q, w_s, E, N, offsets, perm_tok, rows, out, out_dt, ldo,
                            workspace, ws_bytes, status, 0, 0, stream);
}

moe_status moe_grouped_gemm_i8_expire_wait(const void *x_q, const float *x_s, int x_rows, int K, long long ldx,
                                           const void *w_q, const float *w_s, int E, int N, const int32_t *offsets,
                                           const int32_t *perm_tok, int rows, void *out, moe_dtype out_dt, long long ldo,
                                           void *workspace, size_t ws_bytes, uint32_t *status, int role, uint32_t wait_ns,
                                           moe_stream stream)
{
    if (!hook_ok(role, wait_ns)) return MOE_ERR_INVALID_ARG;
    return product<PRODUCT>(x_q, x_s, x_rows, K, ldx, w_q, w_s, w_q, w_s, E, N, offsets, perm_tok, rows, out, out_dt, ldo,
                            workspace, ws_bytes, status, role, wait_ns, stream);
}

moe_status moe_gemm_i8(const void *x_q, const float *x_s, int T, int K, long long ldx, const void *w_q, const float *w_s,
                       int N, void *out, moe_dtype out_dt, long long ldo, void *workspace, size_t ws_bytes,
                       uint32_t *status, moe_stream stream)
{
    return moe_grouped_gemm_i8(x_q, x_s, T, K, ldx, w_q, w_s, 1, N, nullptr, nullptr, T, out, out_dt, ldo, workspace,
                               ws_bytes, status, stream);
}

moe_status moe_gate_up_i8(const void *x_q, const float *x_s, int x_rows, int d, long long ldx, const void *wg_q,
                          const float *wg_s, const void *wu_q, const float *wu_s, int E, int F, const int32_t *offsets,
                          const int32_t *perm_tok, int rows, void *h, moe_dtype h_dt, long long ldh, void *workspace,
                          size_t ws_bytes, uint32_t *status, moe_stream stream)
{
    return product<GATEUP>(x_q, x_s, x_rows, d, ldx, wg_q, wg_s, wu_q, wu_s, E, F, offsets, perm_tok, rows, h, h_dt, ldh,
                           workspace, ws_bytes, status, 0, 0, stream);
}

moe_status moe_gate_up_i8_expire_wait(const void *x_q, const float *x_s, int x_rows, int d, long long ldx, const void *wg_q,
                                      const float *wg_s, const void *wu_q, const float *wu_s, int E, int F,
                                      const int32_t *offsets, const int32_t *perm_tok, int rows, void *h, moe_dtype h_dt,
                                      long long ldh, void *workspace, size_t ws_bytes, uint32_t *status, int role,
                                      uint32_t wait_ns, moe_stream stream)
{
    if (!hook_ok(role, wait_ns)) return MOE_ERR_INVALID_ARG;
    return product<GATEUP>(x_q, x_s, x_rows, d, ldx, wg_q, wg_s, wu_q, wu_s, E, F, offsets, perm_tok, rows, h, h_dt, ldh,
                           workspace, ws_bytes, status, role, wait_ns, stream);
}

}  // extern "C"
