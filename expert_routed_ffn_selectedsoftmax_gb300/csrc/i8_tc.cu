// i8_tc.cu -- products of int8 matrices on the tensor cores (tcgen05, TMA, TMEM): dense,
// grouped by expert with ragged sizes, and the gate/up pair with SwiGLU behind it.
//
//   y[r,n] = (sum_i cx[r,i] cw[n,i]) sx[r] sw[n]
//
// sm_103a has no 8-bit integer MMA.  An int8 code is exact in fp16 and a product of two
// in fp32, so the sums run on kind::f16 and are whole numbers, exact up to 2^24.
//
// Weights are the MMA's rows.  They are read as int8 (TMA), and converter warps -- one
// TMEM lane, that is one weight row, to a thread -- turn 64 codes at a time into fp16 and
// store them into tensor memory, where the MMA takes its A operand: the widened weights
// touch neither HBM nor shared memory.  Tokens are the columns:
//   tiled     128 of them, as fp16 rows that convert_rows_kernel has written (in group
//             order, so it gathers too), by TMA; 256 weight rows a tile (two MMAs of 128
//             rows share the tokens), or 128 of W_gate and the same of W_up;
//   few rows  32, read as int8 and widened into shared memory by the same warps; 128
//             weight rows a tile (or of both); two CTAs an SM.  Few tiles split the
//             reduction over a cluster, whose partial sums meet in distributed shared
//             memory.
// A stage of the reduction is 128 x 128 codes of weights: 64 columns of two tiles, or 128
// of one.  Weights and tokens have rings of their own, as the converters are done with
// the former long before the MMAs are with the latter.
//
// Warp 0 loads weights, warp 3 tokens (one warp for both issued its loads in 930 clocks a
// stage, where the MMAs take 512), warps 1 and 2 multiply a weight tile each, the last 8
// warps convert, four of them a stage, and warps 4.. (4 or 16) write the output.  A
// thread of these holds an output channel; a token's values lie along the warp.
//
// Every wait is bounded (2 s).  Where one gives up, the rows of the CTA's remaining
// tiles are written as NaN, and the status word says so if the caller passed one.
#include <type_traits>

#include "fp8b_tc.cuh"
#include "i8.h"

namespace moe {
namespace i8 {

using namespace sm100;
using fp8b::bar_wait;
using fp8b::elect_one;
using fp8b::Groups;
using fp8b::load_groups;
using fp8b::scan_groups;
using fp8b::Tile;
using fp8b::tile_at;
using fp8b::tma_gather4;
using fp8b::tma_load_3d;

namespace {

constexpr int M = 128;                       // weight rows of an MMA
constexpr int kUnitCols = 32;                // TMEM columns of 64 codes as fp16
constexpr int kStageCols = 2 * kUnitCols;    // ... of a stage's weights
constexpr int kStaging = 2048;
constexpr int kConvWarps = 8;                // two groups of four, which take the stages in turn

template <int MODE, bool FEW> struct Cfg {
    static constexpr int NW = (MODE == GATEUP || !FEW) ? 2 : 1;    // weight tiles of a stage
    static constexpr int BK = NW == 2 ? 64 : 128;
    static constexpr int NT = FEW ? 32 : 128;                      // tokens of a tile
    static constexpr int ROWS = MODE == PRODUCT ? NW * M : M;      // output channels of a tile
    static constexpr int W_BYTES = NW * M * BK;                    // 16 KB
    static constexpr int X_BYTES = NT * BK * (FEW ? 1 : 2);
    static constexpr int WS = FEW ? (MODE == GATEUP ? 5 : 4) : 5;  // stages of the weights' ring
    static constexpr int XS = FEW ? 4 : 6;                         // ... of the tokens'
    static constexpr int NA = FEW ? (MODE == GATEUP ? 2 : 3) : 4;  // converted stages in flight
    static constexpr int XF_BYTES = FEW ? NT * BK * 2 : 0;         // widened tokens of one
    static constexpr int ND = FEW ? 2 : 1;                         // accumulators
    static constexpr int D_COLS = NW * NT;
    static constexpr int A_COL = ND * D_COLS;
    static constexpr int TMEM_COLS = FEW ? 256 : 512;
    static constexpr int EPI = FEW ? 4 : 16;                       // output warps
    static constexpr int THREADS = 128 + 32 * (EPI + kConvWarps);
    static constexpr size_t XRING = (size_t)WS * W_BYTES;
    static constexpr size_t XF = XRING + (size_t)XS * X_BYTES;
    static constexpr size_t STAGING = XF + (size_t)NA * XF_BYTES;  // (tiled: kStaging bytes an output warp)
    static constexpr size_t CTL = STAGING + (FEW ? 0 : (size_t)EPI * kStaging);
    static_assert(A_COL + NA * kStageCols <= TMEM_COLS, "tensor memory");
    static_assert(!FEW || (size_t)NT * NW * M * 4 <= XRING, "split partial sums reuse the weights' ring");
};
constexpr int kMaxW = 5, kMaxX = 6, kMaxA = 4, kTable = 32;

template <int EPI, int TOK> struct alignas(16) Ctl {
    uint64_t wfull[kMaxW], wempty[kMaxW], xfull[kMaxX], xempty[kMaxX], cfull[kMaxA], cempty[kMaxA], dfull[2], dempty[2], drain[2];
    uint64_t never;                          // nothing arrives here (test hook)
    uint32_t tmem_base;
    int abort_flag;
    alignas(16) float sx[EPI][TOK];          // each output warp's token scales
    Groups g;
    Tile tiles[kTable];                      // this CTA's first tiles (each role asks for them in turn)
};
template <int MODE, bool FEW> using CtlOf = Ctl<Cfg<MODE, FEW>::EPI, FEW ? 32 : 64>;
template <int MODE, bool FEW> constexpr size_t smem_bytes() { return 1024 + Cfg<MODE, FEW>::CTL + sizeof(CtlOf<MODE, FEW>); }
static_assert(smem_bytes<PRODUCT, false>() <= 232448 && smem_bytes<GATEUP, false>() <= 232448, "shared memory per CTA");
static_assert(smem_bytes<PRODUCT, true>() <= 115712 && smem_bytes<GATEUP, true>() <= 115712, "two CTAs per SM");
// registers a thread after the split at start (setmaxnreg) of the tiled kernel: 28 warps
// launch with 72 each, 2016; 4 x 40 + 8 x 56 + 16 x 88 = 2016
constexpr int kRegsLaunch = 72, kRegsAux = 40, kRegsConv = 56, kRegsEpi = 88;
static_assert(4 * kRegsAux + 8 * kRegsConv + 16 * kRegsEpi <= 28 * kRegsLaunch, "more registers than the block has");

#define MOE_OUTS8(i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
// 16 columns of the warp's TMEM lanes and the wait for them, in one statement (nothing that
// reads the registers moves above it)
__device__ __forceinline__ void tmem_ld16_wait(uint32_t taddr, uint32_t *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : MOE_OUTS8(0), MOE_OUTS8(8)
        : "r"(taddr)
        : "memory");
}

// The sums of the warp's 32 TMEM lanes (channels) as 8 x 8 fragments, and the wait for them
// in the same statement.  64 columns (tokens): v[32 h + 4 j + 2 r + c] of lane l is channel
// 16 h + 8 r + l / 4, token 8 j + 2 (l % 4) + c.
__device__ __forceinline__ void tmem_ld_frags(uint32_t taddr, uint32_t *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : MOE_OUTS8(0), MOE_OUTS8(8), MOE_OUTS8(16), MOE_OUTS8(24), MOE_OUTS8(32), MOE_OUTS8(40), MOE_OUTS8(48), MOE_OUTS8(56)
        : "r"(taddr), "r"(taddr + (16u << 16))
        : "memory");
}
// 32 columns at each of two places: v[32 m + 16 h + 4 j + 2 r + c]
__device__ __forceinline__ void tmem_ld_frags2(uint32_t a, uint32_t b, uint32_t *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%64];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%65];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47}, [%66];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%67];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : MOE_OUTS8(0), MOE_OUTS8(8), MOE_OUTS8(16), MOE_OUTS8(24), MOE_OUTS8(32), MOE_OUTS8(40), MOE_OUTS8(48), MOE_OUTS8(56)
        : "r"(a), "r"(a + (16u << 16)), "r"(b), "r"(b + (16u << 16))
        : "memory");
}
// Four 8 x 8 fragments of 16-bit values, transposed, to the rows that the lanes name:
// lane 8 m + i row i of fragment m, 16 bytes.
__device__ __forceinline__ void store_frags(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(src))
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// this thread's stores: their shared memory has been read / they are complete
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 16 codes -> 16 fp16 values, in order: q ^ 0x80 = q + 128 in the significand of 1024,
// minus 1152, both exact.
__device__ __forceinline__ void widen16(const uint4 v, uint32_t *o)
{
    const uint32_t w[4] = {v.x ^ 0x80808080u, v.y ^ 0x80808080u, v.z ^ 0x80808080u, v.w ^ 0x80808080u};
    const __half2 off = __half2half2(__ushort_as_half(0x6480));   // 1152
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = __byte_perm(w[i], 0x64646464u, 0x4140), hi = __byte_perm(w[i], 0x64646464u, 0x4342);
        const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&lo), off);
        const __half2 b = __hsub2(*reinterpret_cast<const __half2 *>(&hi), off);
        o[2 * i] = *reinterpret_cast<const uint32_t *>(&a);
        o[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&b);
    }
}
__device__ __forceinline__ bool expires(const Params &p, Role role) { return p.expire_ns && p.expire_role == role; }
// Byte offset of 16-byte piece c of row r in a TMA tile whose rows are BK bytes long
// (64- or 128-byte swizzle).
template <int BK> __device__ __forceinline__ int piece_at(int r, int c)
{
    return r * BK + ((BK == 64 ? c ^ ((r >> 1) & 3) : c ^ (r & 7)) << 4);
}

// Lane l holds channel l's values of 8 tokens, two of bf16 to a word; afterwards it holds
// token l % 8's values of channels 8 (l / 8) .. + 7: a transpose, lane bit by lane bit.
__device__ __forceinline__ void turn8(uint32_t (&w)[4], int lane)
{
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & 4 ? w[q] : w[q + 2], 4);
        if (lane & 4) w[q] = got;
        else w[q + 2] = got;
    }
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & 2 ? w[q] : w[q + 1], 2);
        if (lane & 2) w[q] = got;
        else w[q + 1] = got;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, w[q], 1);
        w[q] = lane & 1 ? __byte_perm(got, w[q], 0x7632) : __byte_perm(w[q], got, 0x5410);
    }
}
// The same of 4 tokens in fp32: token l % 4's values of channels 4 (l / 4) .. + 3.
__device__ __forceinline__ void turn4(uint32_t (&w)[4], int lane)
{
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & 2 ? w[q] : w[q + 2], 2);
        if (lane & 2) w[q] = got;
        else w[q + 2] = got;
    }
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & 1 ? w[q] : w[q + 1], 1);
        if (lane & 1) w[q] = got;
        else w[q + 1] = got;
    }
}

template <int MODE>
__device__ __forceinline__ float finish(const Params &p, float a, float b, float sx, float sw0, float sw1)
{
    if (MODE == PRODUCT) return a * sx * sw0;
    const float g = a * sx * sw0, u = b * sx * sw1;
    return p.out_f32 ? swiglu_accurate(g, u) : swiglu_fast(g, u);
}

// The warp's sums of COUNT tokens (a, and for gate/up b) of output channels n0 + lane:
// scaled and stored.  `row`: the first token's output row; `cnt` of the tokens exist.
// Rows on 16-byte boundaries are turned in registers so that a store covers 8 tokens x 64
// bytes (fp32: 4 x 128) in pieces of 16; else a token at a time, an element a lane.
template <int MODE, int COUNT>
__device__ __forceinline__ void store_tokens(const Params &p, const uint32_t *a, const uint32_t *b, long long row, int cnt, int n0,
                                             int lane, const float *sx, float sw0, float sw1)
{
    const auto value = [&](int q) { return finish<MODE>(p, __uint_as_float(a[q]), __uint_as_float(b[q]), sx[q], sw0, sw1); };
    if (!p.out_vec) {
#pragma unroll
        for (int q = 0; q < COUNT; ++q)
            if (q < cnt && n0 + lane < p.N) store_out(p, row + q, n0 + lane, value(q));
    } else if (p.out_f32) {
        const int n = n0 + (lane >> 2) * 4;
        float *o = static_cast<float *>(p.out) + (row + (lane & 3)) * p.ldo + n;
#pragma unroll
        for (int q = 0; q < COUNT; q += 4) {
            if (q >= cnt) break;
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(value(q + j));
            turn4(w, lane);
            if (q + (lane & 3) < cnt && n < p.N) *reinterpret_cast<uint4 *>(o + q * p.ldo) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
        const int n = n0 + (lane >> 3) * 8;
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + (row + (lane & 7)) * p.ldo + n;
#pragma unroll
        for (int q = 0; q < COUNT; q += 8) {
            if (q >= cnt) break;
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = fp8b::bf16x2(value(q + 2 * j), value(q + 2 * j + 1));
            turn8(w, lane);
            if (q + (lane & 7) < cnt && n < p.N) *reinterpret_cast<uint4 *>(o + q * p.ldo) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// Staged rows of CHANNELS values (16-byte piece c of row t at c ^ (t % 8)) to `rows` of TOKENS output
// rows, CHANNELS threads: 16 bytes at a time where the rows allow, else an element a thread.
template <typename T, int CHANNELS, int TOKENS>
__device__ __forceinline__ void store_staged(T *o, long long ldo, const uint8_t *stg, int tid, int rows, int left, bool vec)
{
    constexpr int V = 16 / (int)sizeof(T);
    if (vec) {
#pragma unroll
        for (int i = 0; i < TOKENS * 8 / CHANNELS; ++i) {
            const int q = tid + i * CHANNELS, t = q >> 3, ch = (q & 7) * V;
            if (t < rows && ch < left) *reinterpret_cast<uint4 *>(o + t * ldo + ch) = *reinterpret_cast<const uint4 *>(stg + piece_at<128>(t, q & 7));
        }
    } else if (tid < left) {
#pragma unroll 4
        for (int t = 0; t < rows; ++t) o[t * ldo + tid] = *reinterpret_cast<const T *>(stg + piece_at<128>(t, tid / V) + (tid % V) * sizeof(T));
    }
}
__device__ __forceinline__ void pair_barrier(int pair) { asm volatile("bar.sync %0, 64;" ::"r"(1 + pair) : "memory"); }

template <int MODE, bool FEW, bool SPLIT>
__global__ void __launch_bounds__((Cfg<MODE, FEW>::THREADS), FEW ? 2 : 1)
product_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w0,
               const __grid_constant__ CUtensorMap tm_w1, const __grid_constant__ CUtensorMap tm_out, const Params p)
{
    using C = Cfg<MODE, FEW>;
    constexpr int NW = C::NW, BK = C::BK, NT = C::NT, WS = C::WS, XS = C::XS, NA = C::NA;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    auto &c = *reinterpret_cast<CtlOf<MODE, FEW> *>(smem + C::CTL);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = p.E;

    if (threadIdx.x == 0) {
        for (int s = 0; s < WS; ++s) { mbar_init(&c.wfull[s], 1); mbar_init(&c.wempty[s], 4); }
        for (int s = 0; s < XS; ++s) { mbar_init(&c.xfull[s], 1); mbar_init(&c.xempty[s], FEW ? 4 : NW); }
        for (int a = 0; a < NA; ++a) { mbar_init(&c.cfull[a], 4); mbar_init(&c.cempty[a], NW); }
        for (int d = 0; d < C::ND; ++d) { mbar_init(&c.dfull[d], NW); mbar_init(&c.dempty[d], C::EPI); }
        for (int w = 0; w < 2; ++w) mbar_init(&c.drain[w], 1);
        mbar_init(&c.never, 1);
        c.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_x)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_w0)) : "memory");
        if (MODE == GATEUP) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_w1)) : "memory");
    }
    if (warp == 3) tmem_alloc(&c.tmem_base, C::TMEM_COLS);
    tc_fence_before();
    // (without offsets nothing up to here reads what the kernel before writes)
    if (p.offsets) pdl_enter();
    load_groups(c.g, p);
    __syncthreads();
    if (warp == 0) scan_groups(c.g, p, NT, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!p.offsets) pdl_enter();

    const uint32_t tmem = c.tmem_base;
    const int S = SPLIT ? p.split : 1;
    const int rank = SPLIT ? (int)cluster_rank() : 0;
    const int first = SPLIT ? blockIdx.x / S : blockIdx.x;
    const int stride = SPLIT ? gridDim.x / S : gridDim.x;
    // (a cluster takes one tile, whatever total the offsets add up to)
    const int total = SPLIT ? min(c.g.total, first + 1) : c.g.total;
    // this CTA's blocks of the reduction
    const int KB = (p.K + BK - 1) / BK;
    const int kb0 = (int)((long long)KB * rank / S), kb1 = (int)((long long)KB * (rank + 1) / S);
    // (a search and two divides a tile)
    if (threadIdx.x < kTable && first + (int)threadIdx.x * stride < total)
        c.tiles[threadIdx.x] = tile_at(c.g, E, first + threadIdx.x * stride, NT);
    __syncthreads();
    auto nth_tile = [&](int i, int t) { return i < kTable ? c.tiles[i] : tile_at(c.g, E, t, NT); };
    volatile int *abort_flag = &c.abort_flag;
    uint32_t issued = 0;   // stages this warp has loaded or multiplied
    bool ok = true;

    if (warp < 4) {
        if (!FEW) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsAux));
        if (warp == 0 || warp == 3) {
            // -------------------------------------------- loads: weights, tokens
            const bool weights = warp == 0;
            const int stages = weights ? WS : XS;
            uint64_t *full = weights ? c.wfull : c.xfull, *empty = weights ? c.wempty : c.xempty;
            uint8_t *ring = smem + (weights ? 0 : C::XRING);
            uint32_t s = 0, phase = 0;
            ok = !expires(p, LOADS) || __all_sync(0xffffffffu, bar_wait(&c.never, 0, abort_flag, p.expire_ns));
            for (int t = first, i = 0; t < total && ok; t += stride, ++i) {
                const Tile tile = nth_tile(i, t);
                const int n0 = tile.nt * C::ROWS;
                int4 tok = make_int4(0, 0, 0, 0);
                const int gathers = FEW && p.perm_tok && !weights ? (tile.cnt + 3) / 4 : 0;
                if (FEW && lane < gathers) {
                    int v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = source_row(p, tile.row0 + min(4 * lane + q, tile.cnt - 1));
                    tok = make_int4(v[0], v[1], v[2], v[3]);
                }
                const uint32_t bytes = weights ? C::W_BYTES : gathers ? gathers * 4 * BK : C::X_BYTES;
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = __all_sync(0xffffffffu, bar_wait(&empty[s], phase ^ 1u, abort_flag));
                    if (!ok) break;
                    uint8_t *at = ring + s * (weights ? C::W_BYTES : C::X_BYTES);
                    if (elect_one()) {
                        mbar_expect_tx(&full[s], bytes);
                        if (weights) {
                            tma_load_3d(at, &tm_w0, &full[s], kb * BK, n0, tile.e);
                            if (MODE == GATEUP) tma_load_3d(at + M * BK, &tm_w1, &full[s], kb * BK, n0, tile.e);
                        } else if (!gathers) {
                            tma_load_2d(at, &tm_x, &full[s], kb * BK, tile.row0);
                        }
                    }
                    __syncwarp();
                    if (FEW && lane < gathers) tma_gather4(at + lane * 4 * BK, &tm_x, &full[s], kb * BK, tok);
                    ++issued;
                    if (++s == (uint32_t)stages) { s = 0; phase ^= 1u; }
                }
            }
            if (!ok) {
                if (lane == 0) flag_status(p.status, kDevTimeout);
                c.abort_flag = 1;
            }
        } else if (warp <= NW) {
            // -------------------------------------------- multiply: a weight tile to a warp
            const bool leader = elect_one();
            const int w = warp - 1;
            const uint32_t tokens = smem_u32(smem + (FEW ? C::XF : C::XRING));
            uint32_t it = 0;
            for (int t = first, i = 0; t < total && ok; t += stride, ++i) {
                const Tile tile = nth_tile(i, t);
                // (N: as many columns as the tile has tokens, in sixteens)
                const uint32_t idesc = idesc_f16_mn(1, M, (tile.cnt + 15) & ~15);
                const int db = i % C::ND;
                const uint32_t d = tmem + db * C::D_COLS + w * NT;
                ok = bar_wait(&c.dempty[db], ((i / C::ND) & 1u) ^ 1u, abort_flag);
                for (int kb = kb0; kb < kb1 && ok; ++kb, ++it) {
                    const uint32_t s = it % XS, a = it % NA;
                    ok = (FEW || bar_wait(&c.xfull[s], (it / XS) & 1u, abort_flag)) &&
                         bar_wait(&c.cfull[a], (it / NA) & 1u, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t dx = sw128_desc(tokens + (FEW ? a * C::XF_BYTES : s * C::X_BYTES));
                    const uint32_t at = tmem + C::A_COL + a * kStageCols + (NW == 2 ? w * kUnitCols : 0);
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            umma_f16_ts(d, at + kk * 8, desc_step(dx, (kk / 4) * NT * 128 + (kk % 4) * 32), idesc, kb != kb0 || kk != 0);
                        if (!FEW) umma_commit(&c.xempty[s]);
                        umma_commit(&c.cempty[a]);
                        if (kb == kb1 - 1) umma_commit(&c.dfull[db]);
                    }
                    __syncwarp();
                }
            }
            if (!ok) {
                if (leader) flag_status(p.status, kDevTimeout);
                c.abort_flag = 1;
            }
            issued = it;
        }
    } else if (warp >= 4 + C::EPI) {
        // ------------------------------------------------ convert
        if (!FEW) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConv));
        // Warps of a group of four take every second stage: a thread row `row` of both
        // weight tiles, or all of its row, and a piece or two of the tokens.
        const int tid = (threadIdx.x - 128 - 32 * C::EPI) & 127, group = (warp - 4 - C::EPI) >> 2;
        const int quad = warp & 3, row = quad * 32 + lane;
        const uint32_t mine = tmem + ((uint32_t)(quad * 32) << 16) + C::A_COL;
        uint32_t it = 0;
        ok = !expires(p, CONVERT) || __all_sync(0xffffffffu, bar_wait(&c.never, 0, abort_flag, p.expire_ns));
        for (int t = first; t < total && ok; t += stride) {
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                if ((it & 1u) != (uint32_t)group) continue;
                const uint32_t s = it % WS, a = it % NA, sx = it % XS;
                ok = __all_sync(0xffffffffu, bar_wait(&c.wfull[s], (it / WS) & 1u, abort_flag) &&
                                                 bar_wait(&c.cempty[a], ((it / NA) & 1u) ^ 1u, abort_flag));
                if (!ok) break;
                tc_fence_after();
                const uint8_t *sw = smem + s * C::W_BYTES;
                const uint32_t at = mine + a * kStageCols;
#pragma unroll
                for (int u = 0; u < 2; ++u) {   // 64 codes: a row of tile u, or half u of a row
                    uint4 v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        v[q] = *reinterpret_cast<const uint4 *>(sw + (NW == 2 ? u * M * BK : 0) + piece_at<BK>(row, (NW == 2 ? 0 : 4 * u) + q));
                    if (u == 1) {   // the stage has been read
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&c.wempty[s]);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t o[16];
                        widen16(v[2 * h], o);
                        widen16(v[2 * h + 1], o + 8);
                        tmem_st16(at + u * kUnitCols + h * 16, o);
                    }
                }
                if (FEW) {
                    ok = __all_sync(0xffffffffu, bar_wait(&c.xfull[sx], (it / XS) & 1u, abort_flag));
                    if (!ok) break;
                    const uint8_t *xs = smem + C::XRING + sx * C::X_BYTES;
                    uint8_t *xf = smem + C::XF + a * C::XF_BYTES;
                    constexpr int PIECES = BK / 16, EACH = NT * PIECES / 128;
#pragma unroll
                    for (int j = 0; j < EACH; ++j) {
                        const int q = tid + j * 128, xr = q / PIECES, xp = q % PIECES;
                        uint32_t h[8];
                        widen16(*reinterpret_cast<const uint4 *>(xs + piece_at<BK>(xr, xp)), h);
                        uint8_t *to = xf + (xp >> 2) * NT * 128;
                        *reinterpret_cast<uint4 *>(to + piece_at<128>(xr, (xp & 3) * 2)) = make_uint4(h[0], h[1], h[2], h[3]);
                        *reinterpret_cast<uint4 *>(to + piece_at<128>(xr, (xp & 3) * 2 + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&c.xempty[sx]);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.cfull[a]);
            }
        }
        if (!ok) {
            if (lane == 0) flag_status(p.status, kDevTimeout);
            c.abort_flag = 1;
        }
    } else {
        // ------------------------------------------------ output
        if (!FEW) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
        const int ew = warp - 4, quarter = warp & 3, part = ew >> 2;
        const int chan = quarter * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
        // (once false, no more waits: the remaining rows become NaN)
        ok = !expires(p, SUMS) || __all_sync(0xffffffffu, bar_wait(&c.never, 0, abort_flag, p.expire_ns));
        for (int t = first, i = 0; t < total; t += stride, ++i) {
            const Tile tile = nth_tile(i, t);
            const int db = i % C::ND;
            const uint32_t d = lane_base + db * C::D_COLS;
            // output channel (tiled PRODUCT: `part` is the weight tile and a half of the
            // tokens; GATEUP: a quarter of them)
            constexpr int TOK = FEW ? NT : MODE == GATEUP ? 32 : 64;
            const int tok0 = FEW ? 0 : (MODE == GATEUP ? part : part & 1) * TOK;
            const int n = tile.nt * C::ROWS + (MODE == PRODUCT ? (part >> 1) * M : 0) + chan;
            float sw0 = 0.f, sw1 = 0.f;
            if (FEW) {
                const long long wn = (long long)tile.e * p.N + min(n, p.N - 1);
                sw0 = __ldg(p.w_s[0] + wn);
                if (MODE == GATEUP) sw1 = __ldg(p.w_s[1] + wn);
            }
            float *sx = c.sx[ew];
            __syncwarp();
            for (int l = lane; l < TOK; l += 32)
                sx[l] = tok0 + l < tile.cnt ? __ldg(p.x_s + source_row(p, tile.row0 + tok0 + l)) : 0.f;
            __syncwarp();
            ok = ok && __all_sync(0xffffffffu, bar_wait(&c.dfull[db], (i / C::ND) & 1u, abort_flag));
            if (!ok) {
                // (the other roles may have left their loops: this warp reports too)
                if (lane == 0) flag_status(p.status, kDevTimeout);
                c.abort_flag = 1;
            }
            tc_fence_after();
            auto done_reading = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.dempty[db]);
            };
            if constexpr (SPLIT) {
                // every MMA of this CTA has completed: the ring holds the partial sums
                // from here on, [token][matrix][channel]
                float *part_sum = reinterpret_cast<float *>(smem) + chan;
#pragma unroll 1
                for (int i0 = 0; i0 < tile.cnt; i0 += 16) {
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        uint32_t v[16];
                        if (ok) tmem_ld16_wait(d + w * NT + i0, v);
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            if (i0 + q < tile.cnt) part_sum[((i0 + q) * NW + w) * M] = ok ? __uint_as_float(v[q]) : 0.f;
                    }
                }
                break;   // one tile per cluster
            } else if constexpr (FEW) {
#pragma unroll 1
                for (int i0 = 0; i0 < tile.cnt; i0 += 16) {
                    uint32_t v[NW][16];
                    if (ok) {
#pragma unroll
                        for (int w = 0; w < NW; ++w) tmem_ld16_wait(d + w * NT + i0, v[w]);
                    } else {
#pragma unroll
                        for (int q = 0; q < 16; ++q) v[0][q] = v[NW - 1][q] = 0x7fffffffu;
                    }
                    if (i0 + 16 >= tile.cnt) done_reading();
                    store_tokens<MODE, 16>(p, v[0], v[NW - 1], tile.row0 + i0, tile.cnt - i0, n - lane, lane, sx + i0, sw0, sw1);
                }
            } else {
                // all of the warp's sums go into registers first: the accumulator is the
                // next tile's from then on
                constexpr int H = MODE == GATEUP ? 16 : 32;   // registers of 16 channels
                const uint32_t from = d + (MODE == GATEUP ? 0 : (part >> 1) * NT) + tok0;
                uint32_t v[64];
                if (!ok) {
#pragma unroll
                    for (int q = 0; q < 64; ++q) v[q] = 0x7fffffffu;
                } else {
                    if (MODE == GATEUP) tmem_ld_frags2(from, from + NT, v);
                    else tmem_ld_frags(from, v);
                }
                done_reading();
                // v[h H + 4 j + 2 r + q]: channel 16 h + 8 r + lane / 4, token 8 j + 2 (lane % 4) + q
                float sw[NW][4];
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const long long at = (long long)tile.e * p.N + min(n - lane + f * 8 + (lane >> 2), p.N - 1);
                    sw[0][f] = __ldg(p.w_s[0] + at);
                    sw[NW - 1][f] = __ldg(p.w_s[NW - 1 < 1 || MODE == PRODUCT ? 0 : 1] + at);
                }
                auto value = [&](int j, int f, int q) {   // octet of tokens, octet of channels, token of a pair
                    const int i = (f >> 1) * H + 4 * j + 2 * (f & 1) + q;
                    const float s = sx[8 * j + 2 * (lane & 3) + q];
                    return finish<MODE>(p, __uint_as_float(v[i]), __uint_as_float(v[(i + 32) & 63]), s, sw[0][f], sw[NW - 1][f]);
                };
                const long long row0 = tile.row0 + tok0;
                const int rows = tile.cnt - tok0;
                if (p.out_f32) {
                    // the warp's 32 channels of 16 tokens at a time
                    uint8_t *stg = smem + C::STAGING + ew * kStaging;
#pragma unroll
                    for (int rd = 0; rd < TOK / 16; ++rd) {
                        if (rd * 16 >= rows) break;
                        if (lane == 0) bulk_wait_read();
                        __syncwarp();
#pragma unroll
                        for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                            for (int f = 0; f < 4; ++f)
#pragma unroll
                                for (int q = 0; q < 2; ++q) {
                                    const int tr = 8 * jj + 2 * (lane & 3) + q, ch = f * 8 + (lane >> 2);
                                    *reinterpret_cast<float *>(stg + piece_at<128>(tr, ch >> 2) + (ch & 3) * 4) = value(2 * rd + jj, f, q);
                                }
                        if (p.out_vec && rows - rd * 16 >= 16) {
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                if (n < p.N) tma_store_2d(&tm_out, stg, n, (int)row0 + rd * 16);
                                bulk_commit();
                            }
                        } else {
                            __syncwarp();
                            float *o = static_cast<float *>(p.out) + (row0 + rd * 16) * p.ldo + n - lane;
                            store_staged<float, 32, 16>(o, p.ldo, stg, lane, min(rows - rd * 16, 16), p.N - (n - lane), p.out_vec);
                        }
                    }
                } else {
                    // the pair's 64 channels of 32 tokens at a time
                    uint8_t *stg = smem + C::STAGING + (ew >> 1) * 2 * kStaging;
                    const int half = ew & 1, n0 = n - lane - half * 32;
#pragma unroll
                    for (int rd = 0; rd < TOK / 32; ++rd) {
                        if (rd * 32 >= rows) break;
                        if (half == 0 && lane == 0) bulk_wait_read();
                        pair_barrier(ew >> 1);
#pragma unroll
                        for (int jj = 0; jj < 4; ++jj) {
                            const int tr = 8 * jj + (lane & 7), j = 4 * rd + jj;
                            uint32_t w[4];
#pragma unroll
                            for (int f = 0; f < 4; ++f) w[f] = fp8b::bf16x2(value(j, f, 0), value(j, f, 1));
                            store_frags(smem_u32(stg + piece_at<128>(tr, half * 4 + (lane >> 3))), w[0], w[1], w[2], w[3]);
                        }
                        if (p.out_vec && rows - rd * 32 >= 32) {
                            fence_proxy_async_smem();
                            pair_barrier(ew >> 1);
                            if (half == 0 && lane == 0) {
                                if (n0 < p.N) tma_store_2d(&tm_out, stg, n0, (int)row0 + rd * 32);
                                bulk_commit();
                            }
                        } else {
                            pair_barrier(ew >> 1);
                            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + (row0 + rd * 32) * p.ldo + n0;
                            store_staged<__nv_bfloat16, 64, 32>(o, p.ldo, stg, half * 32 + lane, min(rows - rd * 32, 32), p.N - n0, p.out_vec);
                        }
                    }
                }
            }
        }
        if (!FEW && lane == 0) bulk_wait_all();
    }

    if constexpr (SPLIT) {
        cluster_sync_all();   // every CTA's partial sums are written
        if (first < total && warp >= 4 && warp < 4 + C::EPI) {
            // tokens rank, rank + S, ...: a thread to a channel adds the CTAs' sums in
            // the order of the blocks
            const Tile tile = nth_tile(0, first);
            const int chan = (warp & 3) * 32 + lane, n = tile.nt * C::ROWS + chan;
            const long long wn = (long long)tile.e * p.N + min(n, p.N - 1);
            const float sw0 = __ldg(p.w_s[0] + wn), sw1 = MODE == GATEUP ? __ldg(p.w_s[1] + wn) : 0.f;
            // (a CTA that gave up may still have had loads landing on its sums)
            bool failed = false;
            for (int q = 0; q < S; ++q) failed |= ld_cluster_u32(peer_addr(&c.abort_flag, q)) != 0u;
            // (four tokens in flight where this CTA has more than one)
            auto add_up = [&](auto tokens) {
                constexpr int U = decltype(tokens)::value, kPeers = U == 1 ? 8 : 2;   // (eight reads in flight)
                for (int i0 = rank; i0 < tile.cnt; i0 += U * S) {
                    float v[U][NW];
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int w = 0; w < NW; ++w) v[u][w] = 0.f;
#pragma unroll kPeers
                    for (int q = 0; q < S; ++q) {
                        const uint32_t at = peer_addr(smem, q) + (uint32_t)chan * 4;
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const int l = min(i0 + u * S, tile.cnt - 1);
#pragma unroll
                            for (int w = 0; w < NW; ++w) v[u][w] += ld_cluster_f32(at + (uint32_t)((l * NW + w) * M) * 4);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int l = i0 + u * S;
                        if (l < tile.cnt && n < p.N) {
                            const float bad = __uint_as_float(0x7fffffffu);
                            store_out(p, tile.row0 + l, n,
                                      finish<MODE>(p, failed ? bad : v[u][0], failed ? bad : v[u][NW - 1], c.sx[warp - 4][l], sw0, sw1));
                        }
                    }
                }
            };
            if (tile.cnt <= S) add_up(std::integral_constant<int, 1>());
            else add_up(std::integral_constant<int, 4>());
        }
        cluster_sync_all();   // no CTA leaves while a peer reads its shared memory
    } else {
        __syncthreads();
    }
    if (*abort_flag) {
        // A role gave up, and nothing says that the others have waited for what was
        // issued: loads land before the CTA exits, MMAs end before TMEM is freed.
        volatile int no_abort = 0;
        if (warp == 0 || warp == 3) {
            const uint32_t stages = warp == 0 ? WS : XS;
            for (uint32_t j = issued >= stages ? issued - stages : 0; j < issued; ++j)
                bar_wait(warp == 0 ? &c.wfull[j % stages] : &c.xfull[j % stages], (j / stages) & 1u, &no_abort, 1000000ull);
        } else if (warp <= NW && issued > 0) {
            if (elect_one()) umma_commit(&c.drain[warp - 1]);
            bar_wait(&c.drain[warp - 1], 0, &no_abort);
        }
        __syncthreads();
    }
    if (warp == 3) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// x's codes as fp16 rows in group order, 16 codes a thread of `kConvertRows` rows (all
// asked for before the first is widened); a token index out of range gives a row of zeros.
constexpr int kConvertThreads = 256, kConvertRows = 4;
struct ConvertLayout { int lanes_log2, col_blocks; };   // threads of a CTA along a row, CTAs along it
__global__ void __launch_bounds__(kConvertThreads)
convert_rows_kernel(const Params p, const ConvertLayout l, uint4 *__restrict__ xf)
{
    pdl_enter();
    const int pieces = p.K / 16, lanes = 1 << l.lanes_log2, each = kConvertThreads >> l.lanes_log2;
    const long long band = blockIdx.x / l.col_blocks;
    const int c = (int)(blockIdx.x - band * l.col_blocks) * lanes + (threadIdx.x & (lanes - 1));
    const long long r0 = band * (kConvertRows * each) + (threadIdx.x >> l.lanes_log2);
    if (c >= pieces) return;
    uint4 v[kConvertRows];
#pragma unroll
    for (int u = 0; u < kConvertRows; ++u) {
        const long long r = r0 + u * each;
        v[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= p.rows) continue;
        const long long src = p.perm_tok ? __ldg(p.perm_tok + r) : r;
        if (src >= 0 && src < p.x_rows) v[u] = __ldg(reinterpret_cast<const uint4 *>(p.x_q + src * p.ldx) + c);
    }
#pragma unroll
    for (int u = 0; u < kConvertRows; ++u) {
        const long long r = r0 + u * each;
        if (r >= p.rows) continue;
        uint32_t o[8];
        widen16(v[u], o);
        uint4 *to = xf + (r * pieces + c) * 2;
        to[0] = make_uint4(o[0], o[1], o[2], o[3]);
        to[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// ------------------------------------------------------------------- host
// [n, rows, cols] of `type` (n = 0: [rows, cols]), rows `ld` bytes apart, box {box_cols, box_rows}
bool make_map(CUtensorMap *m, CUtensorMapDataType type, const void *base, int n, int rows, int cols, long long ld,
              uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle)
{
    auto enc = tc::encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)n};
    const cuuint64_t strides[2] = {(cuuint64_t)ld, (cuuint64_t)ld * (cuuint64_t)rows};
    const cuuint32_t box[3] = {box_cols, box_rows, 1};
    const cuuint32_t one[3] = {1, 1, 1};
    return enc(m, type, n ? 3 : 2, const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, bool FEW, bool SPLIT>
cudaError_t launch_variant(const CUtensorMap &x, const CUtensorMap &w0, const CUtensorMap &w1, const CUtensorMap &out, const Params &p,
                           long long tiles, int num_sms, cudaStream_t stream)
{
    using C = Cfg<MODE, FEW>;
    static PerDeviceFlag done;
    const int dev = current_device();
    auto *kern = product_kernel<MODE, FEW, SPLIT>;
    constexpr size_t smem = smem_bytes<MODE, FEW>();
    if (!done.done(dev)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        done.mark(dev);
    }
    if (SPLIT)
        return launch_pdl_cluster(kern, dim3((unsigned)(tiles * p.split)), dim3(C::THREADS), smem, stream, p.split, x, w0, w1, out, p);
    const long long most = (long long)num_sms * (FEW ? 2 : 1);
    return launch_pdl(kern, dim3((unsigned)(tiles < most ? tiles : most)), dim3(C::THREADS), smem, stream, x, w0, w1, out, p);
}

// Most tiles there can be: an expert with r rows has (r - 1) / rows_per_tile + 1, so as
// many experts as possible with rows, and the rest of the rows in whole tiles.
long long most_tiles(const Params &p, int rows_per_tile)
{
    const long long experts = p.E < p.rows ? p.E : p.rows;
    return ((p.rows - experts) / rows_per_tile + experts) * p.n_tiles;
}

template <int MODE, bool FEW>
bool weight_maps(const Params &p, CUtensorMap *w0, CUtensorMap *w1)
{
    using C = Cfg<MODE, FEW>;
    const auto swizzle = C::BK == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    const auto map = [&](CUtensorMap *m, const void *w) {
        return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, p.E, p.N, p.K, p.K, C::BK, C::ROWS, swizzle);
    };
    if (!map(w0, p.w[0])) return false;
    if (MODE != GATEUP) { *w1 = *w0; return true; }
    return map(w1, p.w[1]);
}

}  // namespace

size_t tiled_workspace(int rows, int K) { return align_up((size_t)rows * K * 2, 256); }

template <int MODE> cudaError_t launch_tiled(const Params &args, void *workspace, cudaStream_t stream)
{
    using C = Cfg<MODE, false>;
    Params p = args;
    const int num_sms = device_sm_count();
    p.n_tiles = ceil_div(p.N, C::ROWS);
    p.split = 1;
    const long long tiles = most_tiles(p, C::NT);
    if (tiles > 0x3fffffffLL) return cudaErrorInvalidValue;
    ConvertLayout l{0, 1};
    while (l.lanes_log2 < 8 && (1 << l.lanes_log2) < p.K / 16) ++l.lanes_log2;
    l.col_blocks = ceil_div(p.K / 16, 1 << l.lanes_log2);
    const int per = kConvertRows * (kConvertThreads >> l.lanes_log2);
    const long long ctas = (long long)ceil_div(p.rows, per) * l.col_blocks;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    const cudaError_t e = launch_pdl(convert_rows_kernel, dim3((unsigned)ctas), dim3(kConvertThreads), 0, stream, p, l,
                                     static_cast<uint4 *>(workspace));
    if (e != cudaSuccess) return e;
    CUtensorMap mx, mw0, mw1;
    if (!make_map(&mx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, workspace, 0, p.rows, p.K, (long long)p.K * 2, C::BK, C::NT,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
        !weight_maps<MODE, false>(p, &mw0, &mw1))
        return cudaErrorInvalidValue;
    CUtensorMap mout = mx;   // (not used where rows are not on 16-byte boundaries)
    if (p.out_vec && !make_map(&mout, p.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.out, 0, p.rows,
                               p.N, p.ldo * (p.out_f32 ? 4 : 2), p.out_f32 ? 32 : 64, p.out_f32 ? 16 : 32, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    return launch_variant<MODE, false, false>(mx, mw0, mw1, mout, p, tiles, num_sms, stream);
}

template <int MODE> cudaError_t launch_few(const Params &args, cudaStream_t stream)
{
    using C = Cfg<MODE, true>;
    Params p = args;
    const int num_sms = device_sm_count();
    p.n_tiles = ceil_div(p.N, C::ROWS);
    const long long tiles = most_tiles(p, C::NT);
    if (tiles > 0x3fffffffLL) return cudaErrorInvalidValue;
    // tiles for fewer than half the SMs: split the reduction over a CTA for each SM, at
    // most 8 a tile
    p.split = 1;
    const int KB = ceil_div(p.K, C::BK);
    if (2 * tiles <= num_sms && KB >= 8) {
        const long long each = num_sms / tiles;
        p.split = (int)(each < 8 ? each : 8);
    }
    CUtensorMap mx, mw0, mw1;
    if (!make_map(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.x_q, 0, p.x_rows, p.K, p.ldx, C::BK, p.perm_tok ? 1 : C::NT,
                  C::BK == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B) ||
        !weight_maps<MODE, true>(p, &mw0, &mw1))
        return cudaErrorInvalidValue;
    return p.split > 1 ? launch_variant<MODE, true, true>(mx, mw0, mw1, mx, p, tiles, num_sms, stream)
                       : launch_variant<MODE, true, false>(mx, mw0, mw1, mx, p, tiles, num_sms, stream);
}

template cudaError_t launch_tiled<PRODUCT>(const Params &, void *, cudaStream_t);
template cudaError_t launch_tiled<GATEUP>(const Params &, void *, cudaStream_t);
template cudaError_t launch_few<PRODUCT>(const Params &, cudaStream_t);
template cudaError_t launch_few<GATEUP>(const Params &, cudaStream_t);

}  // namespace i8
}  // namespace moe
