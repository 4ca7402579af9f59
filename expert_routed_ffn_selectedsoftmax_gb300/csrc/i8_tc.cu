// i8_tc.cu -- products of int8 matrices on the tensor cores (tcgen05, TMA, TMEM): dense,
// grouped by expert with ragged sizes, and the gate/up pair with SwiGLU behind it.
//
//   y[r,n] = (sum_i cx[r,i] cw[n,i]) sx[r] sw[n]
//
// sm_103a has no 8-bit integer MMA.  An int8 code is exact in fp16 and a product of two
// in fp32, so the sums run on kind::f16 and are whole numbers, exact up to 2^24; beyond, each
// step of 16 columns may cut off a unit in their last place (8192 x 2048 x 5632's sums of normal
// values stay below; 16384 columns of codes from 100 to 127 came out 5.4e-5 too small).
//
// Weights are the MMA's 128 rows (PRODUCT: of W; GATEUP: 64 of W_gate and the same 64 of
// W_up, 16 of each to the lanes of a warp, so that the warp that writes a channel has both of
// its sums).  They are read as int8 (TMA), and converter warps -- one TMEM lane, that is one
// weight row, to a thread -- widen 128 codes of it at a time to fp16 and store them into
// tensor memory, where the MMA takes its A operand: the widened weights touch neither HBM
// nor shared memory.  Tokens are the columns:
//   tiled     128 of them, as fp16 rows that convert_rows_kernel has written (in group
//             order, so it gathers too), by TMA; one CTA an SM;
//   few rows  32, read as int8 and widened into shared memory by the same warps; two CTAs
//             an SM.
// Accumulators are two, so a tile's output overlaps the next tile's products.  Few tiles
// split the reduction over a cluster, whose CTAs send their partial sums to the one that
// finishes the token (distributed shared memory).
//
// Warp 0 loads weights, warp 3 tokens (one warp for both issued its loads in 930 clocks a
// block of 128 columns' 256 x 64, where the MMAs take 512), warp 1 (tiled: 1 and 2, 64 tokens
// each, 128 us for 8192 x 2048 x 5632 and 141 with one) multiplies, the last 8 warps convert,
// four of them a block in turn, and warps 4.. (4 or 16) write the output.
//
// What bounds it (us, one GB300).  Few rows: the weights' bytes once it runs, and its start and
// end.  Gate/up of 64 experts of 1024 x 512 and 128 x 2 rows takes 16.4; each further block of
// 128 columns adds 1.31, which is 6.4 TB/s, and 6 do not depend on K.  With an SM for each
// tile a block takes 0.39: 1040 clocks to convert, 830 from the MMAs' issue until the buffer
// is free again, three buffers (4096 x 4096 of 128 rows 16.0; rings of 6 and 8 blocks 15.6 and
// 15.9, the output warps as a third converting group 15.9, half blocks in six buffers 18.8, a
// warp of its own for the tokens 22.6).  Tiled: the MMAs, and
// what they share the SM with.  8192 x 2048 x 5632 takes 127 in a graph (1.49 PFLOP/s, 79 % of the
// measured bf16 rate; 136, 74 %, called with new outputs): without the converters' work it takes 120, without the output 120,
// without the tokens' loads 119, and with the MMAs alone 102.  The tensor pipe is busy for
// 72 % of the cycles, and the L2 is at 68 % of its rate.
//
// Every wait is bounded (2 s).  Where one gives up, the rows of the CTA's remaining
// tiles are written as NaN, and the status word says so if the caller passed one.
#include <atomic>
#include <type_traits>

#include "fp8b_tc.cuh"
#include "i8.h"

namespace moe {
namespace i8 {

using namespace sm100;
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
constexpr int BK = kBlock;
constexpr int W_BYTES = M * BK;
constexpr int kBlockCols = BK / 2;           // TMEM columns of a block's weights as fp16
constexpr int kStaging = 2048;
constexpr int kConvWarps = 8;                // two groups of four, which take the blocks in turn
// a CTA's share of a tile's tokens, with the sums of every CTA that splits the reduction (few
// rows: whole turns of the tokens over the CTAs)
constexpr size_t partial_bytes(int tokens) { return (size_t)(tokens + kMaxSplit) * M * 4; }

// The kernels: NT tokens a tile, 128 or (few rows, whole or with a split reduction) 32.  (Tiles
// of 64 tokens, which leave room for 3 blocks of weights and 2 converted, took 0.69 us a block
// where 32 take 0.40.)
template <int NT, bool SPLIT = false> struct Cfg {
    static constexpr bool FEW = NT < 128;
    static constexpr int X_BYTES = NT * BK * (FEW ? 1 : 2);
    static constexpr int WS = FEW && SPLIT ? 3 : 4;                       // blocks of the weights' ring
    static constexpr int NA = FEW ? 3 : 4;                         // converted blocks in flight
    static constexpr int XS = 4;                                   // blocks of the tokens' ring (tiled: block a's
                                                                   // tokens are freed with its converted weights)
    static constexpr int XF_BYTES = FEW ? NT * BK * 2 : 0;         // widened tokens of a block
    static constexpr int A_COL = 2 * NT;                           // (two accumulators before)
    static constexpr int TMEM_COLS = FEW ? 256 : 512;
    static constexpr int MMAS = FEW ? 1 : 2;                       // multiplying warps, each with its share of the tokens
    static constexpr int EPI = FEW ? 4 : 16;                       // output warps
    static constexpr int THREADS = 128 + 32 * (EPI + kConvWarps);
    static constexpr size_t XRING = (size_t)WS * W_BYTES;
    static constexpr size_t XF = XRING + (size_t)XS * X_BYTES;
    static constexpr size_t STAGING = XF + (size_t)NA * XF_BYTES;
    // split: the CTAs' sums of this CTA's tokens, sent as soon as each has them (few rows) or
    // into the rings when all have (tiled).  (Two CTAs an SM also let the next kernel of the
    // stream start beside this one.)
    static constexpr size_t PARTIAL = FEW ? STAGING : 0;
    static constexpr size_t CTL = STAGING + (!FEW ? EPI / 2 * kStaging : SPLIT ? partial_bytes(NT) : 0);
    static_assert(PARTIAL + partial_bytes(NT) <= (FEW ? PARTIAL + partial_bytes(NT) : STAGING), "the rings hold the sums");
    static_assert(A_COL + NA * kBlockCols <= TMEM_COLS, "tensor memory");
    static_assert(WS >= NA && XS >= NA, "a converting group waits for a phase that the other has left");
    static_assert(FEW || XS == NA, "a tiled block's tokens and converted weights share an index");
    static_assert(NT == 128 || NT == 32, "an output warp has 32 tokens");
};
constexpr int kMaxRing = 4, kTable = 32;

template <int EPI> struct alignas(16) Ctl {
    uint64_t wfull[kMaxRing], wempty[kMaxRing], xfull[kMaxRing], xempty[kMaxRing], cfull[kMaxRing], cempty[kMaxRing];
    uint64_t dfull[2], dempty[2], drain[2];
    uint64_t never;                          // nothing arrives here (test hook)
    uint32_t tmem_base;
    int abort_flag;
    uint32_t lost;                           // split: a CTA of the cluster has no sums to send
    alignas(16) float sx[EPI][32], sw[EPI][2][EPI == 4 ? 1 : 32];   // each output warp's scales: tokens', channels' (tiled)
    Groups g;
    Tile tiles[kTable];                      // this CTA's first tiles (each role asks for them in turn)
};
template <int NT> using CtlOf = Ctl<Cfg<NT>::EPI>;
template <int NT, bool SPLIT = false> constexpr size_t smem_bytes() { return 1024 + Cfg<NT, SPLIT>::CTL + sizeof(CtlOf<NT>); }
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<128, true>() <= 232448, "shared memory per CTA");
static_assert(smem_bytes<32>() <= 115712 && smem_bytes<32, true>() <= 115712, "two CTAs per SM");
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

// 32 columns (tokens) of the warp's 32 TMEM lanes (channels) as 8 x 8 fragments, and the
// wait for them in the same statement: v[16 h + 4 j + 2 r + c] of lane l is channel
// 16 h + 8 r + l / 4, token 8 j + 2 (l % 4) + c.
__device__ __forceinline__ void tmem_ld_frags(uint32_t taddr, uint32_t *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : MOE_OUTS8(0), MOE_OUTS8(8), MOE_OUTS8(16), MOE_OUTS8(24)
        : "r"(taddr), "r"(taddr + (16u << 16))
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

// bar_wait with a non-blocking test first: a try_wait takes 130 clocks even of a phase
// that is complete, and the multiplying warp's waits are what its MMAs wait for.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                         unsigned long long timeout_ns = kTimeoutNs)
{
    return mbar_test_wait(bar, parity) || fp8b::bar_wait(bar, parity, abort_flag, timeout_ns);
}

// 4 codes -> 4 fp16 values, in order: q ^ 0x80 = q + 128 in the significand of 1024, minus
// 1152, both exact.
__device__ __forceinline__ void widen4(uint32_t v, uint32_t *o)
{
    const uint32_t w = v ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));   // 1152
    const uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140), hi = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&lo), off);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2 *>(&hi), off);
    o[0] = *reinterpret_cast<const uint32_t *>(&a);
    o[1] = *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ void widen16(const uint4 v, uint32_t *o)
{
    widen4(v.x, o);
    widen4(v.y, o + 2);
    widen4(v.z, o + 4);
    widen4(v.w, o + 6);
}
__device__ __forceinline__ void st_cluster_u32(uint32_t cluster_addr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_v4(uint32_t cluster_addr, const uint32_t *v)
{
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}
// The two halves of a barrier of all threads of the cluster (each warp converged).
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// The block's weight row of TMEM lane 32 `quad` + `lane`.  Gate/up: lanes 0-15 of each warp are
// gate rows, 16-31 the up rows of the same 16 channels.
template <int MODE> __device__ __forceinline__ int weight_row(int quad, int lane)
{
    return MODE == GATEUP ? (lane >> 4) * 64 + quad * 16 + (lane & 15) : quad * 32 + lane;
}
__device__ __forceinline__ bool expires(const Params &p, Role role) { return p.expire_ns && p.expire_role == role; }
// Byte offset of 16-byte piece c of row r in a tile of 128-byte rows (TMA's 128-byte swizzle).
__device__ __forceinline__ int piece_at(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

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

// Two tokens' at once (two fp32 operations an instruction, each rounded as alone).
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
template <int MODE>
__device__ __forceinline__ float2 finish2(const Params &p, const uint32_t *a, const uint32_t *b, float2 sx, float sw0, float sw1)
{
    const float2 g = mul2(mul2(make_float2(__uint_as_float(a[0]), __uint_as_float(a[1])), sx), make_float2(sw0, sw0));
    if (MODE == PRODUCT) return g;
    const float2 u = mul2(mul2(make_float2(__uint_as_float(b[0]), __uint_as_float(b[1])), sx), make_float2(sw1, sw1));
    const float2 e = p.out_f32 ? make_float2(expf(-fabsf(g.x)), expf(-fabsf(g.y))) : make_float2(__expf(-fabsf(g.x)), __expf(-fabsf(g.y)));
    const float2 ge = mul2(g, e);
    return mul2(mul2(make_float2(max_nan(g.x, ge.x), max_nan(g.y, ge.y)), make_float2(reciprocal(1.0f + e.x), reciprocal(1.0f + e.y))), u);
}

// The warp's sums of COUNT tokens (a, and for gate/up b) of output channels n0 + lane:
// scaled and stored.  `row`: the first token's output row; `cnt` of the tokens exist.
// Gate/up: 16 channels, the upper lanes' (as 0-15) of other tokens, so row, cnt and sx are a
// lane's own.
// Rows on 16-byte boundaries are turned in registers so that a store covers whole sectors
// (PRODUCT: 8 tokens x 64 bytes, fp32 4 x 128) in pieces of 16; else a token at a time, an
// element a lane.
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
            if (MODE == PRODUCT && q >= cnt) break;
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
            if (MODE == PRODUCT && q >= cnt) break;
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
            if (t < rows && ch < left) *reinterpret_cast<uint4 *>(o + t * ldo + ch) = *reinterpret_cast<const uint4 *>(stg + piece_at(t, q & 7));
        }
    } else if (tid < left) {
#pragma unroll 4
        for (int t = 0; t < rows; ++t) o[t * ldo + tid] = *reinterpret_cast<const T *>(stg + piece_at(t, tid / V) + (tid % V) * sizeof(T));
    }
}
// Barrier of the four output warps that share their tokens.  (bar.sync is .aligned: the warp
// reconverges first.)
__device__ __forceinline__ void group_barrier(int group)
{
    __syncwarp();
    asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
}

template <int MODE, int NT, bool SPLIT>
__global__ void __launch_bounds__(Cfg<NT>::THREADS, Cfg<NT>::FEW ? 2 : 1)
product_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w0,
               const __grid_constant__ CUtensorMap tm_w1, const __grid_constant__ CUtensorMap tm_out, const Params p)
{
    using C = Cfg<NT, SPLIT>;
    constexpr bool FEW = C::FEW;
    constexpr int WS = C::WS, XS = C::XS, NA = C::NA, ROWS = channels_of_tile(MODE);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    auto &c = *reinterpret_cast<CtlOf<NT> *>(smem + C::CTL);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = p.E;

    if (threadIdx.x == 0) {
        for (int s = 0; s < WS; ++s) { mbar_init(&c.wfull[s], 1); mbar_init(&c.wempty[s], 4); }
        for (int s = 0; s < XS; ++s) { mbar_init(&c.xfull[s], 1); mbar_init(&c.xempty[s], 4); }
        for (int a = 0; a < NA; ++a) { mbar_init(&c.cfull[a], 4); mbar_init(&c.cempty[a], C::MMAS); }
        for (int d = 0; d < 2; ++d) { mbar_init(&c.dfull[d], C::MMAS); mbar_init(&c.dempty[d], C::EPI); }
        for (int w = 0; w < 2; ++w) mbar_init(&c.drain[w], 1);
        mbar_init(&c.never, 1);
        c.abort_flag = 0;
        c.lost = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_x)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_w0)) : "memory");
        if (MODE == GATEUP) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_w1)) : "memory");
    }
    if (warp == 3) tmem_alloc(&c.tmem_base, C::TMEM_COLS);
    tc_fence_before();
    // (without offsets nothing up to the roles reads what the kernel before writes)
    if (p.offsets) pdl_enter();
    load_groups(c.g, p);
    __syncthreads();
    if (warp == 0) scan_groups(c.g, p, NT, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    const uint32_t tmem = c.tmem_base;
    const uint32_t S = SPLIT ? p.split : 1;
    const uint32_t rank = SPLIT ? cluster_rank() : 0;
    const int first = SPLIT ? blockIdx.x / S : blockIdx.x;
    const int stride = SPLIT ? gridDim.x / S : gridDim.x;
    // (a cluster takes one tile, whatever total the offsets add up to)
    const int total = SPLIT ? min(c.g.total, first + 1) : c.g.total;
    // this CTA's blocks of the reduction (at most 2^24 of them, and 8 CTAs)
    const uint32_t KB = (uint32_t)(p.K + BK - 1) / BK;
    const int kb0 = (int)(KB * rank / S), kb1 = (int)(KB * (rank + 1) / S);
    // (a search and two divides a tile)
    if (threadIdx.x < kTable && first + (int)threadIdx.x * stride < total)
        c.tiles[threadIdx.x] = tile_at(c.g, E, first + threadIdx.x * stride, NT);
    __syncthreads();
    if (!p.offsets) pdl_enter();
    // (the CTAs of a cluster may write one another's memory once all have started; tiled: once
    // all have their sums)
    if (SPLIT && FEW) cluster_arrive();
    bool met = false;
    uint8_t *partial = smem + C::PARTIAL;
    auto nth_tile = [&](int i, int t) { return i < kTable ? c.tiles[i] : tile_at(c.g, E, t, NT); };
    volatile int *abort_flag = &c.abort_flag;
    uint32_t issued = 0;   // blocks this warp has loaded or multiplied
    bool ok = true;

    if (warp < 4) {
        if (!FEW) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsAux));
        if (warp == 0) {
            // -------------------------------------------- loads: weights
            uint32_t it = 0;
            ok = !expires(p, LOADS) || __all_sync(0xffffffffu, bar_wait(&c.never, 0, abort_flag, p.expire_ns));
            for (int t = first, i = 0; t < total && ok; t += stride, ++i) {
                const Tile tile = nth_tile(i, t);
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const uint32_t s = it % WS;
                    ok = __all_sync(0xffffffffu, bar_wait(&c.wempty[s], ((it / WS) & 1u) ^ 1u, abort_flag));
                    if (!ok) break;
                    if (elect_one()) {
                        uint8_t *at = smem + s * W_BYTES;
                        mbar_expect_tx(&c.wfull[s], W_BYTES);
                        tma_load_3d(at, &tm_w0, &c.wfull[s], kb * BK, tile.nt * ROWS, tile.e);
                        if (MODE == GATEUP) tma_load_3d(at + ROWS * BK, &tm_w1, &c.wfull[s], kb * BK, tile.nt * ROWS, tile.e);
                    }
                    __syncwarp();
                }
            }
            issued = it;
        } else if (warp == 3) {
            // -------------------------------------------- loads: tokens
            uint32_t it = 0;
            uint64_t *empty = FEW ? c.xempty : c.cempty;
            ok = !expires(p, LOADS) || __all_sync(0xffffffffu, bar_wait(&c.never, 0, abort_flag, p.expire_ns));
            for (int t = first, i = 0; t < total && ok; t += stride, ++i) {
                const Tile tile = nth_tile(i, t);
                int4 tok = make_int4(0, 0, 0, 0);
                const int gathers = FEW && p.perm_tok ? (tile.cnt + 3) / 4 : 0;
                if (FEW && lane < gathers) {
                    int v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = source_row(p, tile.row0 + min(4 * lane + q, tile.cnt - 1));
                    tok = make_int4(v[0], v[1], v[2], v[3]);
                }
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const uint32_t s = it % XS;
                    ok = __all_sync(0xffffffffu, bar_wait(&empty[s], ((it / XS) & 1u) ^ 1u, abort_flag));
                    if (!ok) break;
                    uint8_t *at = smem + C::XRING + s * C::X_BYTES;
                    if (elect_one()) {
                        mbar_expect_tx(&c.xfull[s], gathers ? gathers * 4 * BK : C::X_BYTES);
                        if (!gathers) {
                            tma_load_2d(at, &tm_x, &c.xfull[s], kb * BK, tile.row0);
                            // (a 128-byte row holds 64 columns of fp16)
                            if (!FEW) tma_load_2d(at + NT * 128, &tm_x, &c.xfull[s], kb * BK + 64, tile.row0);
                        }
                    }
                    __syncwarp();
                    if (FEW && lane < gathers) tma_gather4(at + lane * 4 * BK, &tm_x, &c.xfull[s], kb * BK, tok);
                }
            }
            issued = it;
        } else if (warp <= C::MMAS) {
            // -------------------------------------------- multiply
            const bool leader = elect_one();
            constexpr int NM = NT / C::MMAS;
            const int from = (warp - 1) * NM;   // this warp's first token
            const uint32_t tokens = smem_u32(smem + (FEW ? C::XF : C::XRING)) + from * 128;
            uint32_t it = 0;
            for (int t = first, i = 0; t < total && ok; t += stride, ++i) {
                const Tile tile = nth_tile(i, t);
                // (N: as many columns as the tile has tokens, in sixteens)
                const int mine = min(tile.cnt - from, NM);
                const uint32_t idesc = idesc_f16_mn(1, M, (mine + 15) & ~15);
                const int db = i & 1;
                const uint32_t d = tmem + db * NT + from;
                // A lane's waits are its own until the warp votes, behind the issue (ahead of it the
                // vote took up to 1 % of the time): a lane that gave up skips the block, and all
                // of them leave the loop together.
                bool mine_ok = bar_wait(&c.dempty[db], ((i >> 1) & 1u) ^ 1u, abort_flag);
                for (int kb = kb0; kb < kb1 && ok; ++kb, ++it) {
                    const uint32_t a = it % NA;
                    // (the converters have seen the tokens land too)
                    mine_ok = mine_ok && bar_wait(&c.cfull[a], (it / NA) & 1u, abort_flag);
                    if (mine_ok) {
                        tc_fence_after();
                        const uint64_t dx = sw128_desc(tokens + a * (FEW ? C::XF_BYTES : C::X_BYTES));
                        const uint32_t at = tmem + C::A_COL + a * kBlockCols;
                        if (leader) {
                            if (mine > 0)
#pragma unroll
                            for (int kk = 0; kk < BK / 16; ++kk)
                                umma_f16_ts(d, at + kk * 8, desc_step(dx, (kk / 4) * NT * 128 + (kk % 4) * 32), idesc, kb != kb0 || kk != 0);
                            umma_commit(&c.cempty[a]);
                            if (kb == kb1 - 1) umma_commit(&c.dfull[db]);
                        }
                    }
                    ok = __all_sync(0xffffffffu, mine_ok);
                }
            }
            issued = it;
        }
        if (!ok) {
            if (lane == 0) flag_status(p.status, kDevTimeout);
            c.abort_flag = 1;
        }
    } else if (warp >= 4 + C::EPI) {
        // ------------------------------------------------ convert
        if (!FEW) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConv));
        // A group takes every second block: a thread a weight row, and (few rows) two pieces of
        // the tokens.
        const int tid = (threadIdx.x - 128 - 32 * C::EPI) & 127, quad = warp & 3, row = weight_row<MODE>(quad, lane);
        const uint32_t mine = tmem + ((uint32_t)(quad * 32) << 16) + C::A_COL;
        const uint32_t turns = total > first ? (uint32_t)((total - first - 1) / stride + 1) * (uint32_t)(kb1 - kb0) : 0u;
        ok = !expires(p, CONVERT) || __all_sync(0xffffffffu, bar_wait(&c.never, 0, abort_flag, p.expire_ns));
        for (uint32_t it = (warp - 4 - C::EPI) >> 2; it < turns && ok; it += 2) {
            const uint32_t s = it % WS, a = it % NA, sx = it % XS;
            // cempty first: the MMAs of block it - NA are done, so both groups are past block
            // it - WS, and the ring's barriers are at this block's phase.  (Asked first, a
            // barrier that the other group's block is still to complete has the parity of two
            // phases ago, and the wait would pass.)
            ok = __all_sync(0xffffffffu, bar_wait(&c.cempty[a], ((it / NA) & 1u) ^ 1u, abort_flag) &&
                                             bar_wait(&c.wfull[s], (it / WS) & 1u, abort_flag));
            if (!ok) break;
            __syncwarp();
            tc_fence_after();
            const uint8_t *sw = smem + s * W_BYTES;
            const uint32_t at = mine + a * kBlockCols;
#pragma unroll
            for (int u = 0; u < 2; ++u) {   // 64 codes
                uint4 v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const uint4 *>(sw + piece_at(row, 4 * u + q));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t o[16];
                    widen16(v[2 * h], o);
                    widen16(v[2 * h + 1], o + 8);
                    tmem_st16(at + u * 32 + h * 16, o);
                }
            }
            // The block has been read: its codes are in registers that have been used.  (An
            // arrival right behind the loads does not wait for them, and the next block's TMA
            // writes are not ordered with them: rows of the next block's codes came in.)
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.wempty[s]);
            __syncwarp();   // (here and below: the instructions that follow are .aligned)
            ok = __all_sync(0xffffffffu, bar_wait(&c.xfull[sx], (it / XS) & 1u, abort_flag));
            if (!ok) break;
            if (FEW) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int q = tid + j * 128, xr = q >> 3, xp = q & 7;
                    uint8_t *to = smem + C::XF + a * C::XF_BYTES + (xp >> 2) * NT * 128;
                    uint32_t h[8];
                    widen16(*reinterpret_cast<const uint4 *>(smem + C::XRING + sx * C::X_BYTES + piece_at(xr, xp)), h);
                    *reinterpret_cast<uint4 *>(to + piece_at(xr, (xp & 3) * 2)) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4 *>(to + piece_at(xr, (xp & 3) * 2 + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.xempty[sx]);
                __syncwarp();
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.cfull[a]);
        }
        if (!ok) {
            if (lane == 0) flag_status(p.status, kDevTimeout);
            c.abort_flag = 1;
        }
    } else {
        // ------------------------------------------------ output
        if (!FEW) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
        // A warp has the channels of its 32 TMEM lanes (GATEUP: gate and up of 16) and (tiled)
        // 32 of the tokens.
        const int ew = warp - 4, quarter = warp & 3, group = ew >> 2, tok0 = FEW ? 0 : group * 32;
        constexpr int CH = ROWS / 4;   // channels of a warp
        const int chan = quarter * CH, cl = lane % CH;
        const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16) + tok0;
        float *sx = c.sx[ew];
        auto &sw = c.sw[ew];
        // (once false, no more waits: the remaining rows become NaN)
        ok = !expires(p, SUMS) || __all_sync(0xffffffffu, bar_wait(&c.never, 0, abort_flag, p.expire_ns));
        // A tile's scales are asked for a tile ahead, lane l's token and channel l's (two loads,
        // one after the other, where rows are gathered).
        float nx = 0.f, nw[2] = {0.f, 0.f};
        auto enter = [&](int i, int t) {
            if (t >= total) return;
            const Tile next = nth_tile(i, t);
            nx = tok0 + lane < next.cnt ? __ldg(p.x_s + source_row(p, next.row0 + tok0 + lane)) : 0.f;
            const long long at = (long long)next.e * p.N + min(next.nt * ROWS + chan + cl, p.N - 1);
            nw[0] = __ldg(p.w_s[0] + at);
            if (MODE == GATEUP) nw[1] = __ldg(p.w_s[1] + at);
        };
        enter(0, first);
        // 64 channels (from n) of the next 16 tokens (from `row`, `left` exist) out of the staging, by two warps
        auto store_pair = [&](long long row, int n, int left, const uint8_t *st) {
            if (p.out_vec && left >= 16) {
                if ((quarter & 1) == 0 && lane == 0) {
                    if (n < p.N) tma_store_2d(&tm_out, st, n, (int)row);
                    bulk_commit();
                }
            } else if (left > 0) {
                __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + row * p.ldo + n;
                store_staged<__nv_bfloat16, 64, 16>(o, p.ldo, st, (quarter & 1) * 32 + lane, min(left, 16), p.N - n, p.out_vec);
            }
            __syncwarp();
        };
        for (int t = first, i = 0; t < total; t += stride, ++i) {
            const Tile tile = nth_tile(i, t);
            const int db = i & 1, n0 = tile.nt * ROWS + chan;   // the warp's first channel
            const uint32_t d = lane_base + db * NT;
            const int cnt = tile.cnt - tok0;                     // the warp's tokens (none or less: nothing to do)
            const long long row0 = tile.row0 + tok0;
            __syncwarp();
            sx[lane] = nx;
            const float sw0 = nw[0], sw1 = nw[1];
            if constexpr (!FEW) { sw[0][lane] = sw0; sw[1][lane] = sw1; }
            __syncwarp();
            enter(i + 1, t + stride);
            ok = ok && __all_sync(0xffffffffu, bar_wait(&c.dfull[db], (i >> 1) & 1u, abort_flag));
            if (!ok) {
                // (the other roles may have left their loops: this warp reports too)
                if (lane == 0) flag_status(p.status, kDevTimeout);
                c.abort_flag = 1;
                __syncwarp();
            }
            tc_fence_after();
            auto done_reading = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.dempty[db]);
                __syncwarp();
            };
            if constexpr (SPLIT) {
                if constexpr (FEW) {
                    cluster_wait();
                    met = true;
                    // token l's sums go to CTA l % S, which finishes it: [token l / S][CTA][weight row]
                    uint32_t to = 0, at = (uint32_t)weight_row<MODE>(quarter, lane) * 4 + rank * (M * 4);
#pragma unroll 1
                    for (int i0 = 0; i0 < cnt; i0 += 16) {
                        uint32_t v[16];
                        __syncwarp();
                        if (ok) tmem_ld16_wait(d + i0, v);
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            if (i0 + q < cnt) st_cluster_u32(peer_addr(partial, to) + at, ok ? v[q] : 0x7fffffffu);
                            if (++to == S) { to = 0; at += S * M * 4; }
                        }
                    }
                } else {
                    cluster_sync_all();
                    met = true;
                    if (!ok && lane < S) st_cluster_u32(peer_addr(&c.lost, lane), 1u);
                    // NT / S neighbouring tokens to each CTA: [CTA][four tokens][weight row][token]
                    const uint32_t share = NT / S;
#pragma unroll 1
                    for (int i0 = 0; i0 < min(cnt, 32) && ok; i0 += 16) {
                        uint32_t v[16];
                        __syncwarp();
                        tmem_ld16_wait(d + i0, v);
                        const uint32_t l = tok0 + i0;
                        const uint32_t at = peer_addr(partial, l / share) +
                                            ((rank * share + l % share) / 4 * M + weight_row<MODE>(quarter, lane)) * 16;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (i0 + 4 * q < cnt) st_cluster_v4(at + q * M * 16, v + 4 * q);
                    }
                    __syncwarp();
                }
                break;   // one tile per cluster
            } else if constexpr (FEW) {
#pragma unroll 1
                for (int i0 = 0; i0 < cnt; i0 += 16) {
                    uint32_t v[16];
                    __syncwarp();
                    if (ok) {
                        tmem_ld16_wait(d + i0, v);
                    } else {
#pragma unroll
                        for (int q = 0; q < 16; ++q) v[q] = 0x7fffffffu;
                    }
                    if (i0 + 16 >= cnt) done_reading();
                    if constexpr (MODE == GATEUP) {
                        // (the lower lanes finish tokens 0-7 of the sixteen, the upper 8-15)
                        const bool upper = lane >= 16;
                        uint32_t g[8], u[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? v[q] : v[8 + q], 16);
                            g[q] = upper ? got : v[q];
                            u[q] = upper ? v[8 + q] : got;
                        }
                        const int l = i0 + (upper ? 8 : 0);
                        store_tokens<MODE, 8>(p, g, u, row0 + l, cnt - l, n0, cl, sx + l, sw0, sw1);
                    } else {
                        store_tokens<MODE, 16>(p, v, v, row0 + i0, cnt - i0, n0, lane, sx + i0, sw0, sw1);
                    }
                }
            } else {
                uint32_t v[32];
                if (cnt > 0) {   // (the whole group)
                    if (ok) {
                        tmem_ld_frags(d, v);
                    } else {
#pragma unroll
                        for (int q = 0; q < 32; ++q) v[q] = 0x7fffffffu;
                    }
                }
                done_reading();
                if (cnt <= 0) continue;
                // Two warps' channels, staged in the pair's 2 KB as rows of 128 bytes; a warp's
                // share of the values goes out by TMA where its tokens are all there.
                const int pair = quarter >> 1, half = quarter & 1;
                uint8_t *stg = smem + C::STAGING + group * 2 * kStaging, *st = stg + pair * kStaging;
                constexpr int OCTETS = CH / 8;   // of the warp's channels
                auto values = [&](int j, int f) {   // two tokens' of an octet of tokens, an octet of channels
                    const uint32_t *a = v + (f >> 1) * 16 + 4 * j + 2 * (f & 1);
                    return finish2<MODE>(p, a, MODE == GATEUP ? a + 16 : a, *reinterpret_cast<const float2 *>(sx + 8 * j + 2 * (lane & 3)),
                                         sw[0][8 * f + (lane >> 2)], sw[1][8 * f + (lane >> 2)]);
                };
                auto packed = [&](int j, int f) {
                    const float2 x = values(j, f);
                    return fp8b::bf16x2(x.x, x.y);
                };
                // The staging's rows have left (read by the TMA stores of lanes 0, or by these
                // warps): it may be written.  / It has been written.
                auto staging_free = [&] {
                    if (lane == 0) bulk_wait_read();
                    group_barrier(group);
                };
                auto staged = [&] {
                    fence_proxy_async_smem();
                    group_barrier(group);
                };
                if (p.out_f32) {
                    // 32 channels: of one warp and 8 tokens (PRODUCT), of two and 16 (each sends 8)
                    constexpr int T = MODE == GATEUP ? 2 : 1;   // octets of tokens at a time
                    uint8_t *own = st + half * (kStaging / 2);
                    const int np = MODE == GATEUP ? n0 - half * 16 : n0;
#pragma unroll
                    for (int j0 = 0; j0 < 4; j0 += T) {
                        if (j0 * 8 >= cnt) break;   // (the group)
                        if (MODE == GATEUP) {
                            staging_free();
                        } else {
                            if (lane == 0) bulk_wait_read();
                            __syncwarp();
                        }
#pragma unroll
                        for (int j = 0; j < T; ++j)
#pragma unroll
                            for (int f = 0; f < OCTETS; ++f) {
                                const float2 x = values(j0 + j, f);
                                const int tr = 2 * (lane & 3), ch = (MODE == GATEUP ? half * 16 : 0) + f * 8 + (lane >> 2);
                                uint8_t *to = (MODE == GATEUP ? st + j * (kStaging / 2) : own) + (ch & 3) * 4;
                                *reinterpret_cast<float *>(to + piece_at(tr, ch >> 2)) = x.x;
                                *reinterpret_cast<float *>(to + piece_at(tr + 1, ch >> 2)) = x.y;
                            }
                        if (MODE == GATEUP) {
                            staged();
                        } else {
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        const int t0 = j0 * 8 + (MODE == GATEUP ? half * 8 : 0), left = cnt - t0;
                        if (p.out_vec && left >= 8) {
                            if (lane == 0) {
                                if (np < p.N) tma_store_2d(&tm_out, own, np, (int)row0 + t0);
                                bulk_commit();
                            }
                        } else if (left > 0) {
                            float *o = static_cast<float *>(p.out) + (row0 + t0) * p.ldo + np;
                            store_staged<float, 32, 8>(o, p.ldo, own, lane, min(left, 8), p.N - np, p.out_vec);
                        }
                        __syncwarp();
                    }
                } else if constexpr (MODE == PRODUCT) {
                    // two warps' 64 channels of 16 tokens at a time
                    const int np = n0 - half * 32;
#pragma unroll
                    for (int j0 = 0; j0 < 4; j0 += 2) {
                        if (j0 * 8 >= cnt) break;   // (the group)
                        staging_free();
#pragma unroll
                        for (int j = j0; j < j0 + 2; ++j) {
                            uint32_t w[4];
#pragma unroll
                            for (int f = 0; f < 4; ++f) w[f] = packed(j, f);
                            store_frags(smem_u32(st + piece_at(8 * (j - j0) + (lane & 7), half * 4 + (lane >> 3))), w[0], w[1], w[2], w[3]);
                        }
                        staged();
                        store_pair(row0 + j0 * 8, np, cnt - j0 * 8, st);
                    }
                } else {
                    // four warps' 64 channels of all 32 tokens, 16 for each pair to send
                    staging_free();
#pragma unroll
                    for (int j0 = 0; j0 < 4; j0 += 2) {
                        uint32_t w[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m) w[m] = packed(j0 + (m >> 1), m & 1);
                        store_frags(smem_u32(stg + (j0 >> 1) * kStaging + piece_at(8 * (lane >> 4) + (lane & 7), quarter * 2 + ((lane >> 3) & 1))),
                                    w[0], w[1], w[2], w[3]);
                    }
                    staged();
                    store_pair(row0 + pair * 16, n0 - chan, cnt - pair * 16, st);
                }
            }
        }
        if (!FEW && lane == 0) bulk_wait_all();
    }

    if constexpr (SPLIT) {
        __syncwarp();
        if (FEW) {
            if (!met) cluster_wait();
        } else if (!met) {
            cluster_sync_all();
        }
        cluster_sync_all();   // every CTA's partial sums have arrived
        if (first < total && warp >= 4 && warp < 4 + C::EPI) {
            // A thread to a channel adds the CTAs' sums of this CTA's tokens in the order of the
            // blocks.
            const Tile tile = nth_tile(0, first);
            const int tid = threadIdx.x - 128, chan = tid & (ROWS - 1), n = tile.nt * ROWS + chan;
            constexpr int NW = M / ROWS, AT = C::EPI * 32 / ROWS;   // sums of a channel; tokens (tiled: fours) at a time
            const long long wn = (long long)tile.e * p.N + min(n, p.N - 1);
            const float sw0 = __ldg(p.w_s[0] + wn), sw1 = MODE == GATEUP ? __ldg(p.w_s[1] + wn) : 0.f;
            if constexpr (FEW) {
                // tokens rank, rank + S, ... (a CTA that gave up sent NaN)
                for (int own = tid / ROWS, l = rank + own * S; l < tile.cnt; own += AT, l += AT * S) {
                    const float *from = reinterpret_cast<const float *>(partial) + own * S * M + chan;
                    float v[NW];
#pragma unroll
                    for (int w = 0; w < NW; ++w) v[w] = 0.f;
#pragma unroll 8
                    for (uint32_t q = 0; q < S; ++q)
#pragma unroll
                        for (int w = 0; w < NW; ++w) v[w] += from[q * M + w * ROWS];
                    if (n < p.N) store_out(p, tile.row0 + l, n, finish<MODE>(p, v[0], v[NW - 1], c.sx[warp - 4][l], sw0, sw1));
                }
            } else {
                // (a CTA that gave up said so: loads may still have come into the rings)
                const int share = NT / S, from = rank * share;
                const bool lost = c.lost;
                for (int four = tid / ROWS; four < share / 4 && from + 4 * four < tile.cnt; four += AT) {
                    const float4 *at = reinterpret_cast<const float4 *>(partial) + four * M + chan;
                    float4 v[NW];
#pragma unroll
                    for (int w = 0; w < NW; ++w) v[w] = at[w * ROWS];
                    for (uint32_t q = 1; q < S; ++q)
#pragma unroll
                        for (int w = 0; w < NW; ++w) {
                            const float4 x = at[q * (share / 4) * M + w * ROWS];
                            v[w] = make_float4(v[w].x + x.x, v[w].y + x.y, v[w].z + x.z, v[w].w + x.w);
                        }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // (32 tokens' scales with each group of four warps)
                        const int l = from + 4 * four + i;
                        const auto of = [&](const float4 &x) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; };
                        const float y = finish<MODE>(p, lost ? __uint_as_float(0x7fffffffu) : of(v[0]), of(v[NW - 1]), c.sx[l / 32 * 4][l % 32], sw0, sw1);
                        if (l < tile.cnt && n < p.N) store_out(p, tile.row0 + l, n, y);
                    }
                }
            }
        }
        __syncthreads();
    } else {
        __syncthreads();
    }
    if (*abort_flag) {
        // A role gave up, and nothing says that the others have waited for what was
        // issued: loads land before the CTA exits, MMAs end before TMEM is freed.
        volatile int no_abort = 0;
        if (warp == 0 || warp == 3) {
            const uint32_t depth = warp == 0 ? WS : XS;
            for (uint32_t j = issued >= depth ? issued - depth : 0; j < issued; ++j)
                bar_wait(warp == 0 ? &c.wfull[j % depth] : &c.xfull[j % depth], (j / depth) & 1u, &no_abort, 1000000ull);
        } else if (warp <= C::MMAS && issued > 0) {
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

// x's codes as fp16 rows in group order, 8 codes a thread (16 bytes written: a warp's stores
// are whole sectors); a token index out of range gives a row of zeros.  One piece a thread, and
// as many threads as that takes: 192 rows of 2048 columns and their product 12.9 us (several
// rows a thread, all asked for at once: 2 13.2, 4 14.1, 8 16.3), 8192 rows 126.4 (127.0, 127.1,
// 131.2); 128 threads a CTA 132.0, as CTAs start too slowly.
constexpr int kConvertThreads = 256;
struct ConvertLayout { int lanes_log2, col_blocks; };   // threads of a CTA along a row, CTAs along it
__global__ void __launch_bounds__(kConvertThreads)
convert_rows_kernel(const Params p, const ConvertLayout l, uint4 *__restrict__ xf)
{
    pdl_enter();
    const int pieces = p.K / 8, lanes = 1 << l.lanes_log2;
    const long long band = blockIdx.x / l.col_blocks;
    const int c = (int)(blockIdx.x - band * l.col_blocks) * lanes + (threadIdx.x & (lanes - 1));
    const long long r = band * (kConvertThreads >> l.lanes_log2) + (threadIdx.x >> l.lanes_log2);
    if (c >= pieces || r >= p.rows) return;
    const long long src = p.perm_tok ? __ldg(p.perm_tok + r) : r;
    uint2 v = make_uint2(0u, 0u);
    if (src >= 0 && src < p.x_rows) v = __ldg(reinterpret_cast<const uint2 *>(p.x_q + src * p.ldx) + c);
    uint32_t o[4];
    widen4(v.x, o);
    widen4(v.y, o + 2);
    xf[r * pieces + c] = make_uint4(o[0], o[1], o[2], o[3]);
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

template <int MODE, int NT, bool SPLIT> cudaError_t prepare(int dev)
{
    static PerDeviceFlag done;
    if (done.done(dev)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(product_kernel<MODE, NT, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem_bytes<NT, SPLIT>());
    if (e == cudaSuccess) done.mark(dev);
    return e;
}

// Clusters of `S` CTAs of the tiled kernel that run at the same time (0 where that cannot be told).
template <int MODE> int most_clusters(int S)
{
    using C = Cfg<128, true>;
    static std::atomic<int> known[kCachedDevices][kMaxSplit + 1];   // 1 more than the number
    const int dev = current_device();
    if (dev < kCachedDevices)
        if (const int n = known[dev][S].load()) return n - 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(S);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = smem_bytes<128, true>();
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = S;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (prepare<MODE, 128, true>(dev) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, product_kernel<MODE, 128, true>, &cfg) != cudaSuccess || n < 0) {
        (void)cudaGetLastError();
        return 0;
    }
    if (dev < kCachedDevices) known[dev][S].store(n + 1);
    return n;
}

template <int MODE, int NT, bool SPLIT>
cudaError_t launch_variant(const CUtensorMap &x, const CUtensorMap &w0, const CUtensorMap &w1, const CUtensorMap &out, const Params &p,
                           long long tiles, int num_sms, cudaStream_t stream)
{
    using C = Cfg<NT, SPLIT>;
    auto *kern = product_kernel<MODE, NT, SPLIT>;
    constexpr size_t smem = smem_bytes<NT, SPLIT>();
    const cudaError_t e = prepare<MODE, NT, SPLIT>(current_device());
    if (e != cudaSuccess) return e;
    if (SPLIT)
        return launch_pdl_cluster(kern, dim3((unsigned)(tiles * p.split)), dim3(C::THREADS), smem, stream, p.split, x, w0, w1, out, p);
    const long long most = (long long)num_sms * (C::FEW ? 2 : 1);
    return launch_pdl(kern, dim3((unsigned)(tiles < most ? tiles : most)), dim3(C::THREADS), smem, stream, x, w0, w1, out, p);
}

template <int MODE> bool weight_maps(const Params &p, CUtensorMap *w0, CUtensorMap *w1)
{
    const auto map = [&](CUtensorMap *m, const void *w) {
        return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, p.E, p.N, p.K, p.K, BK, channels_of_tile(MODE), CU_TENSOR_MAP_SWIZZLE_128B);
    };
    if (!map(w0, p.w[0])) return false;
    if (MODE != GATEUP) { *w1 = *w0; return true; }
    return map(w1, p.w[1]);
}

}  // namespace

size_t tiled_workspace(int rows, int K) { return align_up((size_t)rows * K * 2, 256); }

template <int MODE> int split_of_tiled(long long tiles, int blocks)
{
    for (int s = kMaxSplit; s > 1; s /= 2)
        if (s * tiles <= device_sm_count() && blocks - blocks / s >= 14 && tiles <= most_clusters<MODE>(s)) return s;
    return 1;
}

template <int MODE> cudaError_t launch_tiled(const Params &args, void *workspace, cudaStream_t stream)
{
    constexpr int NT = 128;
    Params p = args;
    const int num_sms = device_sm_count();
    p.n_tiles = ceil_div(p.N, channels_of_tile(MODE));
    const long long tiles = most_tiles(p.rows, p.E, NT) * p.n_tiles;
    if (tiles > 0x3fffffffLL) return cudaErrorInvalidValue;
    ConvertLayout l{0, 1};
    while ((1 << l.lanes_log2) < kConvertThreads && (1 << l.lanes_log2) < p.K / 8) ++l.lanes_log2;
    l.col_blocks = ceil_div(p.K / 8, 1 << l.lanes_log2);
    const long long ctas = (long long)ceil_div(p.rows, kConvertThreads >> l.lanes_log2) * l.col_blocks;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    const cudaError_t e = launch_pdl(convert_rows_kernel, dim3((unsigned)ctas), dim3(kConvertThreads), 0, stream, p, l,
                                     static_cast<uint4 *>(workspace));
    if (e != cudaSuccess) return e;
    CUtensorMap mx, mw0, mw1;
    if (!make_map(&mx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, workspace, 0, p.rows, p.K, (long long)p.K * 2, 64, NT,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
        !weight_maps<MODE>(p, &mw0, &mw1))
        return cudaErrorInvalidValue;
    CUtensorMap mout = mx;   // (not used where rows are not on 16-byte boundaries)
    if (p.out_vec && !make_map(&mout, p.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.out, 0, p.rows,
                               p.N, p.ldo * (p.out_f32 ? 4 : 2), p.out_f32 ? 32 : 64, p.out_f32 ? 8 : 16, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    p.split = split_of_tiled<MODE>(tiles, ceil_div(p.K, BK));
    return p.split > 1 ? launch_variant<MODE, NT, true>(mx, mw0, mw1, mout, p, tiles, num_sms, stream)
                       : launch_variant<MODE, NT, false>(mx, mw0, mw1, mout, p, tiles, num_sms, stream);
}

template <int MODE> cudaError_t launch_few(const Params &args, cudaStream_t stream)
{
    constexpr int NT = 32;
    Params p = args;
    const int num_sms = device_sm_count();
    p.n_tiles = ceil_div(p.N, channels_of_tile(MODE));
    const long long tiles = most_tiles(p.rows, p.E, NT) * p.n_tiles;
    if (tiles > 0x3fffffffLL) return cudaErrorInvalidValue;
    p.split = split_of(tiles, ceil_div(p.K, BK), num_sms);
    CUtensorMap mx, mw0, mw1;
    if (!make_map(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.x_q, 0, p.x_rows, p.K, p.ldx, BK, p.perm_tok ? 1 : NT,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
        !weight_maps<MODE>(p, &mw0, &mw1))
        return cudaErrorInvalidValue;
    return p.split > 1 ? launch_variant<MODE, NT, true>(mx, mw0, mw1, mx, p, tiles, num_sms, stream)
                       : launch_variant<MODE, NT, false>(mx, mw0, mw1, mx, p, tiles, num_sms, stream);
}

template int split_of_tiled<PRODUCT>(long long, int);
template int split_of_tiled<GATEUP>(long long, int);
template cudaError_t launch_tiled<PRODUCT>(const Params &, void *, cudaStream_t);
template cudaError_t launch_tiled<GATEUP>(const Params &, void *, cudaStream_t);
template cudaError_t launch_few<PRODUCT>(const Params &, cudaStream_t);
template cudaError_t launch_few<GATEUP>(const Params &, cudaStream_t);

}  // namespace i8
}  // namespace moe
