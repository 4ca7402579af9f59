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
// Every unit of conversion is 128 weight rows x 64 columns, and a stage of the ring holds
// two: both weight tiles' (BK = 64), or both halves of one tile's (BK = 128).
//
// Warp 0 loads, warp 1 multiplies, warps 4.. (4 or 8) write the output, the last 8
// convert.  A thread of the output warps holds an output channel; a token's values are
// contiguous over the warp, so they are stored from registers.
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
constexpr int kUnitCols = 32;                // TMEM columns of a converted unit (64 codes as fp16)
constexpr int kConvWarps = 8;                // two groups of four, a unit of each stage to a group

template <int MODE, bool FEW> struct Cfg {
    static constexpr int NW = (MODE == GATEUP || !FEW) ? 2 : 1;    // weight tiles of a stage
    static constexpr int BK = NW == 2 ? 64 : 128;
    static constexpr int NT = FEW ? 32 : 128;                      // tokens of a tile
    static constexpr int ROWS = MODE == PRODUCT ? NW * M : M;      // output channels of a tile
    static constexpr int W_BYTES = NW * M * BK;
    static constexpr int X_BYTES = NT * BK * (FEW ? 1 : 2);
    static constexpr int STAGE = W_BYTES + X_BYTES;
    static constexpr int STAGES = FEW ? (MODE == GATEUP ? 5 : 4) : 6;
    static constexpr int NA = FEW ? 2 : 4;                         // converted stages in flight
    static constexpr int XF_BYTES = FEW ? NT * BK * 2 : 0;         // widened tokens of one
    static constexpr int ND = FEW ? 2 : 1;                         // accumulators
    static constexpr int D_COLS = NW * NT;
    static constexpr int A_COL = ND * D_COLS;
    static constexpr int TMEM_COLS = FEW ? 256 : 512;
    static constexpr int EPI = FEW ? 4 : 16;                       // output warps
    static constexpr int THREADS = 128 + 32 * (EPI + kConvWarps);
    static constexpr size_t RING = (size_t)STAGES * STAGE;
    static constexpr size_t CTL = RING + (size_t)NA * XF_BYTES;
    static_assert(A_COL + NA * 2 * kUnitCols <= TMEM_COLS, "tensor memory");
};
constexpr int kMaxStages = 6, kMaxA = 4, kTable = 32;

struct alignas(16) Ctl {
    uint64_t full[kMaxStages], empty[kMaxStages], cfull[kMaxA], cempty[kMaxA], dfull[2], dempty[2], drain;
    uint64_t never;                          // nothing arrives here (test hook)
    uint32_t tmem_base;
    int abort_flag;
    alignas(16) float sx[16][M];             // each output warp's token scales
    Groups g;
    Tile tiles[kTable];                      // this CTA's first tiles (each role asks for them in turn)
};
template <int MODE, bool FEW> constexpr size_t smem_bytes() { return 1024 + Cfg<MODE, FEW>::CTL + sizeof(Ctl); }
static_assert(smem_bytes<PRODUCT, false>() <= 232448 && smem_bytes<GATEUP, false>() <= 232448, "shared memory per CTA");
static_assert(smem_bytes<PRODUCT, true>() <= 115712 && smem_bytes<GATEUP, true>() <= 115712, "two CTAs per SM");
// registers a thread after the split at start (setmaxnreg) of the tiled kernel: 28 warps
// launch with 72 each, 2016; 4 x 32 + 8 x 56 + 16 x 88 = 1984
constexpr int kRegsLaunch = 72, kRegsAux = 32, kRegsConv = 56, kRegsEpi = 88;
static_assert(4 * kRegsAux + 8 * kRegsConv + 16 * kRegsEpi <= 28 * kRegsLaunch, "more registers than the block has");

#define MOE_OUTS8(i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
// 32 columns of the warp's TMEM lanes and the wait for them, in one statement (nothing that
// reads the registers moves above it)
__device__ __forceinline__ void tmem_ld32_wait(uint32_t taddr, uint32_t *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : MOE_OUTS8(0), MOE_OUTS8(8), MOE_OUTS8(16), MOE_OUTS8(24)
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16_wait(uint32_t taddr, uint32_t *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : MOE_OUTS8(0), MOE_OUTS8(8)
        : "r"(taddr)
        : "memory");
}

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

template <int MODE>
__device__ __forceinline__ float finish(const Params &p, float a, float b, float sx, float sw0, float sw1)
{
    if (MODE == PRODUCT) return a * sx * sw0;
    const float g = a * sx * sw0, u = b * sx * sw1;
    return p.out_f32 ? swiglu_accurate(g, u) : swiglu_fast(g, u);
}

template <int MODE, bool FEW, bool SPLIT>
__global__ void __launch_bounds__((Cfg<MODE, FEW>::THREADS), FEW ? 2 : 1)
product_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w0,
               const __grid_constant__ CUtensorMap tm_w1, const Params p)
{
    using C = Cfg<MODE, FEW>;
    constexpr int NW = C::NW, BK = C::BK, NT = C::NT, STAGES = C::STAGES, NA = C::NA;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Ctl &c = *reinterpret_cast<Ctl *>(smem + C::CTL);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = p.E;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) { mbar_init(&c.full[s], 1); mbar_init(&c.empty[s], FEW ? kConvWarps : 1); }
        for (int a = 0; a < NA; ++a) { mbar_init(&c.cfull[a], kConvWarps); mbar_init(&c.cempty[a], 1); }
        for (int d = 0; d < C::ND; ++d) { mbar_init(&c.dfull[d], 1); mbar_init(&c.dempty[d], C::EPI); }
        mbar_init(&c.drain, 1);
        mbar_init(&c.never, 1);
        c.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_x)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_w0)) : "memory");
        if (MODE == GATEUP) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_w1)) : "memory");
    }
    if (warp == 2) tmem_alloc(&c.tmem_base, C::TMEM_COLS);
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
        if (warp == 0) {
            // -------------------------------------------- loads
            uint32_t it = 0;
            ok = !expires(p, LOADS) || __all_sync(0xffffffffu, bar_wait(&c.never, 0, abort_flag, p.expire_ns));
            for (int t = first, i = 0; t < total && ok; t += stride, ++i) {
                const Tile tile = nth_tile(i, t);
                const int n0 = tile.nt * C::ROWS;
                int4 tok = make_int4(0, 0, 0, 0);
                const int gathers = FEW && p.perm_tok ? (tile.cnt + 3) / 4 : 0;
                if (FEW && lane < gathers) {
                    int v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = source_row(p, tile.row0 + min(4 * lane + q, tile.cnt - 1));
                    tok = make_int4(v[0], v[1], v[2], v[3]);
                }
                // token rows in boxes: only as many as the tile has (tiled)
                constexpr int XBOX = FEW ? NT : 64;
                const int boxes = FEW ? 1 : (tile.cnt + XBOX - 1) / XBOX;
                const uint32_t bytes = C::W_BYTES + (FEW && p.perm_tok ? gathers * 4 * BK : boxes * XBOX * BK * (FEW ? 1 : 2));
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % STAGES;
                    ok = __all_sync(0xffffffffu, bar_wait(&c.empty[s], ((it / STAGES) & 1u) ^ 1u, abort_flag));
                    if (!ok) break;
                    uint8_t *sw = smem + s * C::STAGE, *sx = sw + C::W_BYTES;
                    if (lane == 0) {
                        mbar_expect_tx(&c.full[s], bytes);
                        tma_load_3d(sw, &tm_w0, &c.full[s], kb * BK, n0, tile.e);
                        if (MODE == GATEUP) tma_load_3d(sw + M * BK, &tm_w1, &c.full[s], kb * BK, n0, tile.e);
                        if (!gathers)
                            for (int b = 0; b < boxes; ++b)
                                tma_load_2d(sx + b * XBOX * 128, &tm_x, &c.full[s], kb * BK, tile.row0 + b * XBOX);
                    }
                    __syncwarp();
                    if (FEW && lane < gathers) tma_gather4(sx + lane * 4 * BK, &tm_x, &c.full[s], kb * BK, tok);
                }
            }
            if (!ok) {
                if (lane == 0) flag_status(p.status, kDevTimeout);
                c.abort_flag = 1;
            }
            issued = it;
        } else if (warp == 1) {
            // -------------------------------------------- multiply
            const bool leader = elect_one();
            const uint32_t ring = smem_u32(smem);
            uint32_t it = 0;
            for (int t = first, i = 0; t < total && ok; t += stride, ++i) {
                const Tile tile = nth_tile(i, t);
                // (N: as many columns as the tile has tokens, in sixteens)
                const uint32_t idesc = idesc_f16_mn(1, M, (tile.cnt + 15) & ~15);
                const int db = i % C::ND;
                const uint32_t d = tmem + db * C::D_COLS;
                ok = bar_wait(&c.dempty[db], ((i / C::ND) & 1u) ^ 1u, abort_flag);
                for (int kb = kb0; kb < kb1 && ok; ++kb, ++it) {
                    const int s = it % STAGES, a = it % NA;
                    ok = bar_wait(&c.cfull[a], (it / NA) & 1u, abort_flag);
                    // (the converters have seen the stage land; its fp16 tokens are this warp's to see)
                    if (!FEW) ok = ok && bar_wait(&c.full[s], (it / STAGES) & 1u, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t dx = sw128_desc(FEW ? ring + (uint32_t)C::RING + a * C::XF_BYTES : ring + s * C::STAGE + C::W_BYTES);
                    const uint32_t at = tmem + C::A_COL + a * 2 * kUnitCols;
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk) {
                            const uint64_t dk = desc_step(dx, (kk / 4) * NT * 128 + (kk % 4) * 32);
#pragma unroll
                            for (int w = 0; w < NW; ++w)
                                umma_f16_ts(d + w * NT, at + (NW == 2 ? w * kUnitCols : 0) + kk * 8, dk, idesc, kb != kb0 || kk != 0);
                        }
                        if (!FEW) umma_commit(&c.empty[s]);
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
        const int tid = threadIdx.x - 128 - 32 * C::EPI;
        const int unit = tid >> 7, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t mine = tmem + ((uint32_t)(quad * 32) << 16) + C::A_COL + unit * kUnitCols;
        // this thread's 64 codes: row `row` of weight tile `unit`, or half `unit` of its row
        const int tile_off = NW == 2 ? unit * M * BK : 0, piece0 = NW == 2 ? 0 : unit * 4;
        uint32_t it = 0;
        ok = !expires(p, CONVERT) || __all_sync(0xffffffffu, bar_wait(&c.never, 0, abort_flag, p.expire_ns));
        for (int t = first; t < total && ok; t += stride) {
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % STAGES, a = it % NA;
                ok = __all_sync(0xffffffffu, bar_wait(&c.full[s], (it / STAGES) & 1u, abort_flag) &&
                                                 bar_wait(&c.cempty[a], ((it / NA) & 1u) ^ 1u, abort_flag));
                if (!ok) break;
                tc_fence_after();
                const uint8_t *sw = smem + s * C::STAGE + tile_off;
                uint4 v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const uint4 *>(sw + piece_at<BK>(row, piece0 + q));
                uint4 xv;
                const int xr = NW == 2 ? tid >> 2 : tid >> 3, xp = NW == 2 ? tid & 3 : tid & 7;
                const bool xmine = FEW && (NW == 1 || tid < 128);
                if (xmine) xv = *reinterpret_cast<const uint4 *>(smem + s * C::STAGE + C::W_BYTES + piece_at<BK>(xr, xp));
                if (FEW) {   // the stage has been read
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&c.empty[s]);
                }
                uint32_t o[16];
                widen16(v[0], o);
                widen16(v[1], o + 8);
                tmem_st16(mine + a * 2 * kUnitCols, o);
                uint32_t o2[16];
                widen16(v[2], o2);
                widen16(v[3], o2 + 8);
                tmem_st16(mine + a * 2 * kUnitCols + 16, o2);
                if (xmine) {
                    uint32_t h[8];
                    widen16(xv, h);
                    uint8_t *xf = smem + C::RING + a * C::XF_BYTES + (xp >> 2) * NT * 128;
                    const int q = (xp & 3) * 2;
                    *reinterpret_cast<uint4 *>(xf + piece_at<128>(xr, q)) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4 *>(xf + piece_at<128>(xr, q + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
                }
                tmem_st_wait();
                if (FEW) fence_proxy_async_smem();
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
            const int n = tile.nt * C::ROWS + (MODE == PRODUCT ? (part >> 1) * M : 0) + chan;
            const long long wn = (long long)tile.e * p.N + min(n, p.N - 1);
            const float sw0 = __ldg(p.w_s[0] + wn), sw1 = MODE == GATEUP ? __ldg(p.w_s[1] + wn) : 0.f;
            float *sx = c.sx[ew];
            __syncwarp();
            for (int l = lane; l < tile.cnt; l += 32) sx[l] = __ldg(p.x_s + source_row(p, tile.row0 + l));
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
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        if (i0 + q < tile.cnt && n < p.N)
                            store_out(p, tile.row0 + i0 + q, n,
                                      finish<MODE>(p, __uint_as_float(v[0][q]), __uint_as_float(v[NW - 1][q]), sx[i0 + q], sw0, sw1));
                }
            } else {
                // all of the warp's sums go into registers first: the accumulator is the
                // next tile's from then on
                uint32_t v[64];
                constexpr int TOK = MODE == GATEUP ? 32 : 64;
                const int tok0 = (MODE == GATEUP ? part : part & 1) * TOK;
                if (!ok) {
#pragma unroll
                    for (int q = 0; q < 64; ++q) v[q] = 0x7fffffffu;
                } else {
                    const uint32_t from = d + (MODE == GATEUP ? 0 : (part >> 1) * NT) + tok0;
                    tmem_ld32_wait(from, v);
                    tmem_ld32_wait(from + (MODE == GATEUP ? NT : 32), v + 32);
                }
                done_reading();
                if (n < p.N) {
#pragma unroll
                    for (int q = 0; q < TOK; ++q) {
                        if (tok0 + q >= tile.cnt) break;
                        store_out(p, tile.row0 + tok0 + q, n,
                                  finish<MODE>(p, __uint_as_float(v[q]), __uint_as_float(v[(q + 32) & 63]), sx[tok0 + q], sw0, sw1));
                    }
                }
            }
        }
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
        if (warp == 0) {
            for (uint32_t j = issued >= STAGES ? issued - STAGES : 0; j < issued; ++j)
                bar_wait(&c.full[j % STAGES], (j / STAGES) & 1u, &no_abort, 1000000ull);
        } else if (warp == 1 && issued > 0) {
            if (elect_one()) umma_commit(&c.drain);
            bar_wait(&c.drain, 0, &no_abort);
        }
        __syncthreads();
    }
    if (warp == 2) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// x's codes as fp16 rows in group order, 16 codes a thread; a token index out of range
// gives a row of zeros.
constexpr int kConvertThreads = 256;
__global__ void __launch_bounds__(kConvertThreads)
convert_rows_kernel(const Params p, uint4 *__restrict__ xf)
{
    pdl_enter();
    const int pieces = p.K / 16;
    const long long total = (long long)p.rows * pieces;
    const long long step = (long long)gridDim.x * kConvertThreads;
    constexpr int U = 4;   // pieces in flight
    for (long long i0 = (long long)blockIdx.x * kConvertThreads + threadIdx.x; i0 < total; i0 += U * step) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long i = i0 + u * step;
            v[u] = make_uint4(0u, 0u, 0u, 0u);
            if (i >= total) continue;
            const int r = (int)(i / pieces), c = (int)(i - (long long)r * pieces);
            const int src = p.perm_tok ? __ldg(p.perm_tok + r) : r;
            if (src >= 0 && src < p.x_rows) v[u] = __ldg(reinterpret_cast<const uint4 *>(p.x_q + src * p.ldx) + c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long i = i0 + u * step;
            if (i >= total) continue;
            uint32_t o[8];
            widen16(v[u], o);
            xf[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
            xf[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
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
cudaError_t launch_variant(const CUtensorMap &x, const CUtensorMap &w0, const CUtensorMap &w1, const Params &p,
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
        return launch_pdl_cluster(kern, dim3((unsigned)(tiles * p.split)), dim3(C::THREADS), smem, stream, p.split, x, w0, w1, p);
    const long long most = (long long)num_sms * (FEW ? 2 : 1);
    return launch_pdl(kern, dim3((unsigned)(tiles < most ? tiles : most)), dim3(C::THREADS), smem, stream, x, w0, w1, p);
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
    const long long pieces = (long long)p.rows * (p.K / 16), per = kConvertThreads * 4;
    const long long want = (pieces + per - 1) / per, most = (long long)num_sms * 8;
    cudaError_t e = launch_pdl(convert_rows_kernel, dim3((unsigned)(want < most ? want : most)), dim3(kConvertThreads), 0,
                               stream, p, static_cast<uint4 *>(workspace));
    if (e != cudaSuccess) return e;
    CUtensorMap mx, mw0, mw1;
    if (!make_map(&mx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, workspace, 0, p.rows, p.K, (long long)p.K * 2, C::BK, 64,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
        !weight_maps<MODE, false>(p, &mw0, &mw1))
        return cudaErrorInvalidValue;
    return launch_variant<MODE, false, false>(mx, mw0, mw1, p, tiles, num_sms, stream);
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
    return p.split > 1 ? launch_variant<MODE, true, true>(mx, mw0, mw1, p, tiles, num_sms, stream)
                       : launch_variant<MODE, true, false>(mx, mw0, mw1, p, tiles, num_sms, stream);
}

template cudaError_t launch_tiled<PRODUCT>(const Params &, void *, cudaStream_t);
template cudaError_t launch_tiled<GATEUP>(const Params &, void *, cudaStream_t);
template cudaError_t launch_few<PRODUCT>(const Params &, cudaStream_t);
template cudaError_t launch_few<GATEUP>(const Params &, cudaStream_t);

}  // namespace i8
}  // namespace moe
