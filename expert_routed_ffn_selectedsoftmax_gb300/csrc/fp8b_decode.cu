// fp8b_decode.cu -- the products of fp8b_gemm.cu for few rows per expert
// (decode): the weights are streamed once, and everything else has to fit into
// the time that takes.
//
// The roles of the operands are exchanged: the weights are the MMA's 128 rows
// (TMEM lanes) and up to 32 token rows its columns, so that a block's partial
// sum is 32 columns of TMEM instead of 256, and every lane of the epilogue holds
// an output column with its tokens -- stores of a token are contiguous over the
// warp as they are.  (Tokens as the rows: a decode batch of 4 rows per expert
// kept 4 of 128 lanes busy, and the tile's epilogue and two waves of tiles cost
// more than the weights' time.)
//
// What bounds it: memory.  64 x 2816 x 2048 over 16 experts (92 MB of weights)
// takes 17.1 us, 5.4 TB/s; gate/up of 128 tokens over 64 experts (48 of them with
// rows, 50 MB) 13.9 us, of which 8 us are the weights' and the rest the start
// (launch, group table, first tile) and the last tile's end.
//
// A tile is 128 output columns (PRODUCT: of W; GATEUP: of W_gate and W_up) of
// one expert times up to 32 of its rows.  Warp 0 loads (TMA; token rows in a box
// of 32, or gathered four at a time through perm_tok), warp 1 multiplies, warps
// 2-5 hold the sums.  A token's scale belongs to a column here, so each warp
// lays out the block's 32 factors sx[t] * sw in shared memory and reads them
// back as broadcasts.  Two CTAs share an SM (ring of 3 or 5 stages each), so one
// tile's start and end overlap the other's loads.
//
// Few tiles: the reduction is split over a cluster of up to 8 CTAs (SPLIT), whose
// partial sums meet in distributed shared memory; token t is finished by CTA
// t % split of the cluster, which adds the CTAs' sums in the order of the blocks.
#include "fp8b_tc.cuh"

#include <type_traits>

namespace moe {
namespace fp8b {

namespace {

constexpr int NT = 32;                       // token rows of a tile
constexpr int M = 128, BK = kBlock;
constexpr int W_BYTES = M * BK, X_BYTES = NT * BK;
constexpr int kBuffers = 4;                  // partial sums in TMEM
constexpr int kEpiWarps = 4;
constexpr int kThreads = 64 + 32 * kEpiWarps;

template <int MODE> struct Cfg {
    static constexpr int NW = MODE == GATEUP ? 2 : 1;           // weight matrices
    static constexpr int STAGE = NW * W_BYTES + X_BYTES;
    static constexpr int STAGES = MODE == GATEUP ? 3 : 5;
    static constexpr int TMEM_COLS = kBuffers * NW * NT;        // 128 or 256
    static constexpr size_t RING = (size_t)STAGES * STAGE;
};
constexpr int kMaxStages = 5;

struct alignas(16) Ctl {
    uint64_t full[kMaxStages], empty[kMaxStages], tfull[kBuffers], tempty[kBuffers], drain;
    uint64_t never;                          // nothing arrives here (test hook)
    uint32_t tmem_base;
    int abort_flag;
    uint32_t amax[kEpiWarps][NT];            // GATEUP: each warp's largest |h| per token
    alignas(16) float factor[kEpiWarps][2][NT];   // [warp][matrix][token], read four at a time
    Groups g;
};
template <int MODE> constexpr size_t smem_bytes() { return 1024 + Cfg<MODE>::RING + sizeof(Ctl); }
static_assert(smem_bytes<PRODUCT>() <= 115712 && smem_bytes<GATEUP>() <= 115712, "two CTAs per SM");
static_assert((size_t)NT * 2 * M * 4 <= Cfg<GATEUP>::RING && (size_t)NT * M * 4 <= Cfg<PRODUCT>::RING,
              "split partial sums reuse the ring");

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}
// Wait for the warp's TMEM loads; the registers pass through it, so that
// nothing that reads them moves above it.
__device__ __forceinline__ void tmem_ld_wait32(uint32_t (&v)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void epilogue_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ void store_out(const Params &p, long long r, int n, float v)
{
    if (p.out_f32) static_cast<float *>(p.out)[r * p.ldo + n] = v;
    else static_cast<__nv_bfloat16 *>(p.out)[r * p.ldo + n] = __float2bfloat16_rn(v);
}

template <int MODE, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 2)
decode_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w0,
              const __grid_constant__ CUtensorMap tm_w1, const Params p)
{
    using C = Cfg<MODE>;
    constexpr int NW = C::NW, STAGES = C::STAGES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Ctl &c = *reinterpret_cast<Ctl *>(smem + C::RING);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = p.E;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) { mbar_init(&c.full[s], 1); mbar_init(&c.empty[s], 1); }
        for (int b = 0; b < kBuffers; ++b) { mbar_init(&c.tfull[b], 1); mbar_init(&c.tempty[b], kEpiWarps); }
        mbar_init(&c.drain, 1);
        mbar_init(&c.never, 1);
        c.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_x)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_w0)) : "memory");
        if (MODE == GATEUP)
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_w1)) : "memory");
    }
    if (warp == 1) tmem_alloc(&c.tmem_base, C::TMEM_COLS);
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
    const int kb0 = (int)((long long)p.KB * rank / S), kb1 = (int)((long long)p.KB * (rank + 1) / S);
    volatile int *abort_flag = &c.abort_flag;
    uint32_t issued = 0;   // blocks this warp has loaded or multiplied

    if (warp == 0) {
        // ------------------------------------------------ loads
        uint32_t it = 0;
        bool ok = !expires(p, LOADS) || __all_sync(0xffffffffu, mbar_wait_slow(&c.never, 0, abort_flag, p.expire_ns));
        for (int t = first; t < total && ok; t += stride) {
            const Tile tile = tile_at(c.g, E, t, NT);
            int4 tok = make_int4(0, 0, 0, 0);
            const int gathers = p.perm_tok ? (tile.cnt + 3) / 4 : 0;
            if (lane < gathers) {
                int v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // (an index out of range reads row 0: its row is undefined)
                    v[i] = __ldg(p.perm_tok + tile.row0 + min(4 * lane + i, tile.cnt - 1));
                    if (v[i] < 0 || v[i] >= p.x_rows) v[i] = 0;
                }
                tok = make_int4(v[0], v[1], v[2], v[3]);
            }
            const uint32_t bytes = NW * W_BYTES + (p.perm_tok ? gathers * 4 * BK : X_BYTES);
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % STAGES;
                ok = __all_sync(0xffffffffu, bar_wait(&c.empty[s], ((it / STAGES) & 1u) ^ 1u, abort_flag));
                if (!ok) break;
                uint8_t *sw = smem + s * C::STAGE, *sx = sw + NW * W_BYTES;
                if (lane == 0) {
                    mbar_expect_tx(&c.full[s], bytes);
                    tma_load_3d(sw, &tm_w0, &c.full[s], kb * BK, tile.nt * M, tile.e);
                    if (MODE == GATEUP) tma_load_3d(sw + W_BYTES, &tm_w1, &c.full[s], kb * BK, tile.nt * M, tile.e);
                    if (!p.perm_tok) tma_load_2d(sx, &tm_x, &c.full[s], kb * BK, tile.row0);
                }
                __syncwarp();
                if (lane < gathers) tma_gather4(sx + lane * 4 * BK, &tm_x, &c.full[s], kb * BK, tok);
            }
        }
        if (!ok) {
            if (lane == 0) flag_status(p.status, kDevTimeout);
            c.abort_flag = 1;
        }
        issued = it;
    } else if (warp == 1) {
        // ------------------------------------------------ multiply
        constexpr uint32_t idesc = idesc_e4m3(M, NT);
        const bool leader = elect_one();
        const uint32_t ring = smem_u32(smem);
        uint32_t it = 0;
        bool ok = true;
        for (int t = first; t < total && ok; t += stride) {
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % STAGES;
                const uint32_t b = it % kBuffers;
                ok = bar_wait(&c.tempty[b], ((it / kBuffers) & 1u) ^ 1u, abort_flag) &&
                     bar_wait(&c.full[s], (it / STAGES) & 1u, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const uint64_t dw = sw128_desc(ring + s * C::STAGE), dx = sw128_desc(ring + s * C::STAGE + NW * W_BYTES);
                const uint32_t d = tmem + b * NW * NT;
                if (leader) {
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        const uint64_t da = desc_step(dw, w * W_BYTES);
                        umma_f8<false>(d + w * NT, da, dx, idesc);
#pragma unroll
                        for (int kk = 1; kk < BK / 32; ++kk)
                            umma_f8<true>(d + w * NT, desc_step(da, kk * 32), desc_step(dx, kk * 32), idesc);
                    }
                    umma_commit(&c.tfull[b]);
                    umma_commit(&c.empty[s]);
                }
            }
        }
        if (!ok) {
            if (leader) flag_status(p.status, kDevTimeout);
            c.abort_flag = 1;
        }
        // (the waits' answers are each lane's own, and what follows is the whole warp's)
        issued = __reduce_max_sync(0xffffffffu, it);
    } else {
        // ------------------------------------------------ sums and output
        const int ew = warp - 2, quarter = warp & 3, chan = quarter * 32 + lane;
        uint32_t it = 0;
        // (once false, no more waits: the remaining rows become NaN)
        bool ok = !expires(p, SUMS) || __all_sync(0xffffffffu, mbar_wait_slow(&c.never, 0, abort_flag, p.expire_ns));
        for (int t = first; t < total; t += stride) {
            const Tile tile = tile_at(c.g, E, t, NT);
            // lane l of every warp holds token l's scales
            const float *xs = nullptr;
            if (lane < tile.cnt) {
                const int r = tile.row0 + lane;
                const int src = p.perm_tok ? __ldg(p.perm_tok + r) : r;
                if (src >= 0 && src < p.x_rows) xs = p.x_s + (size_t)src * p.KB;
            }
            const float *ws[2];
#pragma unroll
            for (int w = 0; w < NW; ++w) ws[w] = p.w_s[w] + ((size_t)tile.e * p.NB + tile.nt) * p.KB;
            uint64_t acc[NW][NT / 2];
#pragma unroll
            for (int w = 0; w < NW; ++w)
#pragma unroll
                for (int i = 0; i < NT / 2; ++i) acc[w][i] = 0ull;
            float nx = xs ? __ldg(xs + kb0) : 0.f, nw[2] = {__ldg(ws[0] + kb0), NW == 2 ? __ldg(ws[NW - 1] + kb0) : 0.f};
#pragma unroll 1
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const uint32_t b = it % kBuffers;
                float(&f)[2][NT] = c.factor[ew];
                __syncwarp();   // (the block before has been read)
#pragma unroll
                for (int w = 0; w < NW; ++w) f[w][lane] = nx * nw[w];
                if (kb + 1 < kb1) {
                    nx = xs ? __ldg(xs + kb + 1) : 0.f;
#pragma unroll
                    for (int w = 0; w < NW; ++w) nw[w] = __ldg(ws[w] + kb + 1);
                }
                __syncwarp();
                ok = ok && __all_sync(0xffffffffu, bar_wait(&c.tfull[b], (it / kBuffers) & 1u, abort_flag));
                if (!ok) continue;   // (TMEM that no MMA has written is not read)
                tc_fence_after();
                const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16) + b * NW * NT;
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    uint32_t v[NT];
                    tmem_ld32(base + w * NT, v);
                    tmem_ld_wait32(v);
                    if (w == NW - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&c.tempty[b]);
                    }
#pragma unroll
                    for (int i = 0; i < NT / 4; ++i) {
                        const float4 q = *reinterpret_cast<const float4 *>(&f[w][4 * i]);
                        fma2(acc[w][2 * i], pack2(v[4 * i], v[4 * i + 1]), pack2(__float_as_uint(q.x), __float_as_uint(q.y)));
                        fma2(acc[w][2 * i + 1], pack2(v[4 * i + 2], v[4 * i + 3]), pack2(__float_as_uint(q.z), __float_as_uint(q.w)));
                    }
                }
            }
            if (!ok) {
                // (the other roles may have left their loops: this warp reports too)
                if (lane == 0) flag_status(p.status, kDevTimeout);
                c.abort_flag = 1;
#pragma unroll
                for (int w = 0; w < NW; ++w)
#pragma unroll
                    for (int i = 0; i < NT / 2; ++i) acc[w][i] = 0x7fffffff7fffffffull;
            }
            auto val = [&](int w, int i) { return (i & 1) ? hi2(acc[w][i >> 1]) : lo2(acc[w][i >> 1]); };
            const int n = tile.nt * M + chan;
            if constexpr (SPLIT) {
                // every MMA of this CTA has completed: the ring holds the partial
                // sums from here on, [token][matrix][channel]
                float *part = reinterpret_cast<float *>(smem) + chan;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    if (i >= tile.cnt) break;
#pragma unroll
                    for (int w = 0; w < NW; ++w) part[(i * NW + w) * M] = val(w, i);
                }
                break;   // one tile per cluster
            } else if constexpr (MODE == GATEUP) {
                // (eight tokens at a time, with or without rows: a branch for each
                // would put their exponentials one after the other)
                uint32_t mine = 0u;   // lane l: largest |h| of token l over the warp's channels
#pragma unroll
                for (int i0 = 0; i0 < NT; i0 += 8) {
                    if (i0 >= tile.cnt) break;
                    float h[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        h[i] = swiglu(val(0, i0 + i), val(NW - 1, i0 + i));
                        const uint32_t m = __reduce_max_sync(0xffffffffu, mag_bits(h[i]));
                        if (lane == i0 + i) mine = m;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)   // (h takes the place of its gate sum)
                        acc[0][i0 / 2 + i] = pack2(__float_as_uint(h[2 * i]), __float_as_uint(h[2 * i + 1]));
                }
                c.amax[ew][lane] = mine;
                epilogue_barrier();   // (all four warps take every turn of the tile loop, whatever happened before)
#pragma unroll
                for (int w = 0; w < kEpiWarps; ++w) mine = max(mine, c.amax[w][lane]);
                epilogue_barrier();
                const float s = block_scale(mine), f = code_factor(s);
                if (ew == 0 && lane < tile.cnt) p.h_s[(size_t)(tile.row0 + lane) * p.NB + tile.nt] = s;
                uint8_t *o = p.h_q + (size_t)tile.row0 * p.N + n;
#pragma unroll
                for (int i0 = 0; i0 < NT; i0 += 8) {
                    if (i0 >= tile.cnt) break;
#pragma unroll
                    for (int i = i0; i < i0 + 8; ++i) {
                        const float q = val(0, i) * __shfl_sync(0xffffffffu, f, i);
                        if (i < tile.cnt && n < p.N) o[(size_t)i * p.N] = (uint8_t)e4m3x2(q, 0.f);
                    }
                }
            } else {
#pragma unroll
                for (int i0 = 0; i0 < NT; i0 += 8) {
                    if (i0 >= tile.cnt) break;
#pragma unroll
                    for (int i = i0; i < i0 + 8; ++i)
                        if (i < tile.cnt && n < p.N) store_out(p, tile.row0 + i, n, val(0, i));
                }
            }
        }
    }

    if constexpr (SPLIT) {
        cluster_sync_all();   // every CTA's partial sums are written
        if (first < total && warp >= 2) {
            // tokens rank, rank + S, ...: a thread to a channel adds the CTAs'
            // sums in the order of the blocks
            const Tile tile = tile_at(c.g, E, first, NT);
            const int ew = warp - 2, chan = (warp & 3) * 32 + lane, n = tile.nt * M + chan;
            // (a CTA that gave up may still have had loads landing on its sums)
            bool failed = false;
            for (int q = 0; q < S; ++q) failed |= ld_cluster_u32(peer_addr(&c.abort_flag, q)) != 0u;
            // (four tokens in flight where this CTA has more than one: one after the
            // other, their reads of the other CTAs' memory took longer than the
            // products)
            auto finish = [&](auto tokens) {
                constexpr int U = decltype(tokens)::value, kPeers = U == 1 ? 8 : 2;   // (eight reads in flight)
                for (int i0 = rank, turn = 0; i0 < tile.cnt; i0 += U * S, turn ^= 1) {
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
                            const int i = min(i0 + u * S, tile.cnt - 1);
#pragma unroll
                            for (int w = 0; w < NW; ++w) v[u][w] += ld_cluster_f32(at + (uint32_t)((i * NW + w) * M) * 4);
                        }
                    }
                    if (failed) {
#pragma unroll
                        for (int u = 0; u < U; ++u)
#pragma unroll
                            for (int w = 0; w < NW; ++w) v[u][w] = __uint_as_float(0x7fffffffu);
                    }
                    if constexpr (MODE == GATEUP) {
                        float h[U];
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            h[u] = swiglu(v[u][0], v[u][NW - 1]);
                            const uint32_t m = __reduce_max_sync(0xffffffffu, mag_bits(h[u]));
                            if (lane == 0) c.amax[ew][turn * U + u] = m;
                        }
                        epilogue_barrier();   // (the other turn's places are written next)
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            uint32_t m = 0u;
#pragma unroll
                            for (int w = 0; w < kEpiWarps; ++w) m = max(m, c.amax[w][turn * U + u]);
                            const float s = block_scale(m);
                            const long long r = tile.row0 + i0 + u * S;
                            if (i0 + u * S < tile.cnt) {
                                if (n < p.N) p.h_q[r * p.N + n] = (uint8_t)e4m3x2(h[u] * code_factor(s), 0.f);
                                if (threadIdx.x == 64) p.h_s[r * p.NB + tile.nt] = s;
                            }
                        }
                    } else {
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            if (i0 + u * S < tile.cnt && n < p.N) store_out(p, tile.row0 + i0 + u * S, n, v[u][0]);
                    }
                }
            };
            if (tile.cnt <= S) finish(std::integral_constant<int, 1>());
            else finish(std::integral_constant<int, 4>());
        }
        cluster_sync_all();   // no CTA leaves while a peer reads its shared memory
    } else {
        __syncthreads();
    }
    if (*abort_flag) {
        // A role gave up, and nothing says that the sums' warps have waited for
        // what the others issued (which may have left their loops before): loads
        // land before the CTA exits, MMAs end before TMEM is freed.
        volatile int no_abort = 0;
        if (warp == 0) {
            for (uint32_t j = issued >= STAGES ? issued - STAGES : 0; j < issued; ++j)
                mbar_wait_slow(&c.full[j % STAGES], (j / STAGES) & 1u, &no_abort, 1000000ull);
        } else if (warp == 1 && issued > 0) {
            if (elect_one()) umma_commit(&c.drain);
            mbar_wait_slow(&c.drain, 0, &no_abort, kTimeoutNs);
        }
        __syncthreads();
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

template <int MODE, bool SPLIT>
cudaError_t launch_variant(const CUtensorMap &x, const CUtensorMap &w0, const CUtensorMap &w1, const Params &p,
                           long long tiles, int num_sms, cudaStream_t stream)
{
    static PerDeviceFlag done;
    const int dev = current_device();
    auto *kern = decode_kernel<MODE, SPLIT>;
    constexpr size_t smem = smem_bytes<MODE>();
    if (!done.done(dev)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        done.mark(dev);
    }
    if (SPLIT)
        return launch_pdl_cluster(kern, dim3((unsigned)(tiles * p.split)), dim3(kThreads), smem, stream, p.split, x, w0,
                                  w1, p);
    return launch_pdl(kern, dim3((unsigned)(tiles < 2 * num_sms ? tiles : 2 * num_sms)), dim3(kThreads), smem, stream,
                      x, w0, w1, p);
}

}  // namespace

// Most tiles there can be: an expert with r rows has (r - 1) / NT + 1, so as
// many experts as possible with rows, and the rest of the rows in whole tiles.
static long long most_tiles(const Params &p)
{
    const long long experts = p.E < p.rows ? p.E : p.rows;
    return ((p.rows - experts) / NT + experts) * ceil_div(p.N, M);
}

// Few rows per expert (at most 16 on average over the experts that can have
// any), or so few tiles that each has an SM: beyond, the rows' tiles read the
// weights again too often.  Against the other kernel, us a call (here / there):
// 64 experts of 1024 x 2 x 512, rows per expert 2: 12.1 / 17.8, 16: 15.7 / 21.2,
// 24: 21.2 / 21.3, 64: 27.5 / 22.8; one of 2048 x 5632 (44 column tiles), rows 16:
// 6.1 / 10.3, 96: 7.8 / 10.3, 128: 9.6 / 10.4, 256: 15.9 / 10.5; 4096 x 4096 (32),
// 16: 6.2 / 16.1, 128: 12.1 / 16.4, 192: 17.4 / 16.5.
// The groups' sizes are known on the device only, so the rule goes by the mean.
// Rows of 16 on average, evenly spread | half of them on one expert | all but one
// for each of the others on one (here / there): 64 experts of 512 x 1024 9.9 / 12.0 |
// 12.0 / 11.9 | 12.2 / 12.1, of 2048 x 1024 26.1 / 28.0 | 29.6 / 27.7 | 30.3 / 27.6,
// 16 of 2816 x 2048 18.8 / 20.6 | 24.0 / 20.6 | 22.6 / 20.6 (gate/up 33.2 / 36.2 |
// 42.0 / 35.7 | 39.7 / 35.7): up to 11 % gained at even loads, up to 18 % lost at these.
bool decode_fits(const Params &p, int num_sms)
{
    const long long experts = p.E < p.rows ? p.E : p.rows;
    return p.rows <= 16 * experts || most_tiles(p) <= num_sms;
}

template <int MODE>
cudaError_t launch_decode(const void *x_q, long long ldx, const void *w0, const void *w1, Params p, int num_sms,
                          cudaStream_t stream)
{
    p.n_tiles = ceil_div(p.N, M);
    const long long tiles = most_tiles(p);
    if (tiles > 0x3fffffffLL) return cudaErrorInvalidValue;
    // tiles for fewer than half the SMs: split the reduction over a CTA for each
    // SM, at most 8 a tile (one token, 2048 x 5632 in 44 tiles: 2 CTAs a tile
    // 5.8 us, 4: 6.2, 6: 6.5; 1024 x 2 x 512 of two experts in 8 tiles: 2 CTAs a
    // tile 6.4 us, 4: 5.9, 8: 5.4).  Short reductions stay whole, as the CTAs'
    // meeting costs more than the blocks it saves: a product of 16 tokens and 1024
    // columns takes 4.1 us split and 3.7 whole at K = 512, 5.1 and 4.5 at 896, 5.2
    // and 6.8 at 2048 (one token 3.6 and 4.3 at 1024); gate/up, with two products a
    // block, of one token and F = 512 5.0 and 4.75 at d = 256, 5.3 and 5.6 at 512.
    // More tiles than half the SMs stay whole too: two CTAs a tile take 8.4 us for 7.7
    // at 32 rows x 2048 x 77 tiles, 12.2 for 10.1 at 150 (at K = 6352 and 77 tiles
    // they would win, 17.7 for 20.3).
    p.split = 1;
    if (2 * tiles <= num_sms && p.KB >= (MODE == GATEUP ? 4 : 8)) {
        const long long each = num_sms / tiles;
        p.split = (int)(each < 8 ? each : 8);
        if (p.split > p.KB) p.split = p.KB;
    }
    CUtensorMap mx, mw0, mw1;
    if (!code_map(&mx, x_q, 0, p.x_rows, p.K, ldx, p.perm_tok ? 1 : NT) || !code_map(&mw0, w0, p.E, p.N, p.K, p.K, M))
        return cudaErrorInvalidValue;
    if (MODE != GATEUP) mw1 = mw0;
    else if (!code_map(&mw1, w1, p.E, p.N, p.K, p.K, M)) return cudaErrorInvalidValue;
    return p.split > 1 ? launch_variant<MODE, true>(mx, mw0, mw1, p, tiles, num_sms, stream)
                       : launch_variant<MODE, false>(mx, mw0, mw1, p, tiles, num_sms, stream);
}

template cudaError_t launch_decode<PRODUCT>(const void *, long long, const void *, const void *, Params, int, cudaStream_t);
template cudaError_t launch_decode<GATEUP>(const void *, long long, const void *, const void *, Params, int, cudaStream_t);

}  // namespace fp8b
}  // namespace moe
