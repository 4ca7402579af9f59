// fp8b_gemm.cu -- products of block-scaled fp8 matrices on the tensor cores
// (tcgen05 kind::f8f6f4, TMA, TMEM): dense, grouped by expert with ragged
// sizes, and the grouped gate/up pair with SwiGLU and quantisation behind it.
//
//   y[r,n] = sum_b sx[r,b] sw[n/128,b] P_b[r,n],   P_b[r,n] = sum_{i in block b} cx[r,i] cw[n,i]
//
// with E4M3 codes c, an activation scale per row and 128 columns and a weight
// scale per 128 x 128 block.  The scales change every 128 columns of the
// reduction, so the tensor cores sum one block (four MMAs of K = 32, fp32)
// into a TMEM buffer -- each half of a tile's columns has two, and a warp that
// issues its MMAs -- and the epilogue warps add that partial sum, times the two
// scales, to the row's running fp32 sums in registers while the tensor cores fill
// the half's other buffer and those of the other half.
//
// What bounds it: 8192 x 2048 x 5632 takes 82 us, 2.3 PFLOP/s (a library product
// with one scale for each matrix, which needs no such turns: 51 us).  A block of
// a 128 x 256 tile takes 870 clocks (traced in the kernel), in which its MMAs keep
// the tensor pipe busy for 512 (ncu: 75.9k of 141k active cycles for 148 blocks an
// SM, 54 %; L2 38 %, issue slots 44 %): the rest is the turn of a TMEM buffer --
// commit, wake, read, sums, arrival, wake -- that the other buffers' MMAs do not
// cover, and a tile's end, where its sums are written while the MMAs run at most
// two blocks ahead.  Tried and no faster: CTA pairs (M = 256; 85 us, and ragged
// groups pad more), one issuing warp with N = 256 (89), sixteen epilogue warps
// (98), scalar sums (89), loads of 32 columns in two register buffers (spills; 127).
//
// A tile is 128 rows x 256 columns (PRODUCT), or 128 rows x 128 columns of
// both W_gate and W_up (GATEUP: the epilogue has whole 128-column groups of h,
// so it quantises them without a second pass).  Warp 0 loads by TMA (rows in
// boxes of 32, only as many as the tile has), warps 1 and 2 multiply a column
// half each, warps 4-11 hold the sums: warp w the TMEM lanes of quarter w % 4
// and one half of the columns (128 of them, or 64 of gate and the same 64 of up).
// Calls of few rows take the kernel of fp8b_decode.cu instead.
//
// Rows of a tile past the end of its group are left out of the loads and the
// stores (their lanes of the MMA compute on whatever the buffer holds; rows
// do not mix).  Columns past N and the last block's columns past K are zeros
// by TMA's fill.
//
// Every wait is bounded (2 s).  Where one gives up, the rows of the CTA's
// remaining tiles are written as NaN, and the status word says so if the
// caller passed one.
#include "fp8b_tc.cuh"

namespace moe {
namespace fp8b {

constexpr int BM = 128, BN = 256, BK = kBlock;   // one MMA k-block = one scale block
constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE = A_BYTES + B_BYTES;
constexpr int STAGES = 3;
constexpr int ABOX = 32;                         // rows per A load
constexpr int TMEM_COLS = 512;                   // two partial sums of 256 columns
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;   // warps 0-3: load, multiply, multiply, TMEM
// registers a thread after the split at start (setmaxnreg): the block launches
// with 168 x 12 warps = 2016; 4 warps keep 56 and 8 take 224: 224 + 1792 = 2016
constexpr int kRegsLaunch = 168, kRegsAux = 56, kRegsEpi = 224;
static_assert(4 * kRegsAux + kEpiWarps * kRegsEpi <= (kThreads / 32) * kRegsLaunch, "more registers than the block has");
constexpr int kStaging = 32 * 256;               // bytes per epilogue warp: 256 of each of its rows

constexpr int kTable = 32;

struct alignas(16) Ctl {
    uint64_t full[STAGES], empty[STAGES], tfull[2][2], tempty[2][2], drain[2];   // [buffer][column half]
    uint64_t never;           // nothing arrives here (test hook)
    uint32_t tmem_base;
    int abort_flag;
    Groups g;
    uint32_t amax[2][BM];     // GATEUP: each row's largest |h| per column half
    Tile tiles[kTable];       // this CTA's first tiles (each role asks for them in turn)
};
constexpr size_t kRing = (size_t)STAGES * STAGE;          // then the staging (from a multiple of 1024
constexpr size_t kCtl = kRing + kEpiWarps * kStaging;     // bytes: the stores' swizzle), then Ctl
constexpr size_t kSmem = 1024 + kCtl + sizeof(Ctl);
static_assert(kSmem <= 232448, "shared memory per CTA");

#define MOE_OUTS16(v, i)                                                                                        \
    "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), \
        "=r"(v[i + 7]), "=r"(v[i + 8]), "=r"(v[i + 9]), "=r"(v[i + 10]), "=r"(v[i + 11]), "=r"(v[i + 12]),      \
        "=r"(v[i + 13]), "=r"(v[i + 14]), "=r"(v[i + 15])
// 64 consecutive columns of the warp's 32 TMEM lanes, and the wait for them (one
// statement: nothing that reads the registers can move above the wait)
__device__ __forceinline__ void tmem_ld64_wait(uint32_t taddr, uint32_t (&v)[64])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,"
        "%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : MOE_OUTS16(v, 0), MOE_OUTS16(v, 16), MOE_OUTS16(v, 32), MOE_OUTS16(v, 48)
        : "r"(taddr)
        : "memory");
}
// A tile from shared to global memory; at most the tensor's bounds are written.
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
// 64 bytes of each of the warp's 32 rows (lane l holds row l's) to global
// memory: turned through shared memory so that a store instruction covers 8
// rows x 64 bytes, whole 32-byte sectors, instead of 32 rows x 16 bytes, which
// took longer than the products of a tile (8192 x 2048 x 5632: 178 us against
// 100 us without the stores).  16-byte piece q of row r lies at q ^ (r / 2 % 4),
// so neither side has bank conflicts.  `g`: row 0's bytes; `rows` of the 32 and
// the first `bytes` exist; rows lie at multiples of 16 bytes, and a last piece
// that is not whole is stored by elements of `size` bytes.
__device__ __forceinline__ void store_rows(uint8_t *stg, int lane, const uint4 (&d)[4], uint8_t *g, long long pitch,
                                           int rows, int bytes, int size)
{
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4 *>(stg + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) = d[q];
    __syncwarp();
    const int q = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2);
        const uint4 v = *reinterpret_cast<const uint4 *>(stg + r * 64 + ((q ^ ((r >> 1) & 3)) << 4));
        const int at = q * 16;
        if (r >= rows || at >= bytes) continue;
        uint8_t *o = g + r * pitch + at;
        if (at + 16 <= bytes) {
            *reinterpret_cast<uint4 *>(o) = v;
        } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (at + k * 4 >= bytes) break;
                if (size == 4) {
                    *reinterpret_cast<uint32_t *>(o + k * 4) = w[k];
                } else {
                    *reinterpret_cast<uint16_t *>(o + k * 4) = (uint16_t)w[k];
                    if (at + k * 4 + 2 < bytes) *reinterpret_cast<uint16_t *>(o + k * 4 + 2) = (uint16_t)(w[k] >> 16);
                }
            }
        }
    }
    __syncwarp();
}

// One staged 128-byte piece of each of `rows` rows (16-byte part q of row r at
// q ^ (r % 8)) to rows of any alignment, element by element.
template <typename T>
__device__ __forceinline__ void store_elements(const Params &p, const uint8_t *at, int lane, long long row0, int n, int rows)
{
    constexpr int V = 16 / (int)sizeof(T);   // elements of a 16-byte part
    T *o = static_cast<T *>(p.out) + row0 * p.ldo + n;
#pragma unroll 4
    for (int r = 0; r < rows; ++r)
#pragma unroll
        for (int c = lane; c < 8 * V; c += 32)
            if (n + c < p.N)
                o[r * p.ldo + c] = *reinterpret_cast<const T *>(at + r * 128 + (((c / V) ^ (r & 7)) << 4) + (c % V) * sizeof(T));
}

// EXPIRE: the test hook (p.expire_ns), a variant of its own so that the other
// does not carry it (it took 1.5 % of a prefill's product)
template <int MODE, bool EXPIRE>
__global__ void __launch_bounds__(kThreads, 1)
product_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w0,
               const __grid_constant__ CUtensorMap tm_w1, const __grid_constant__ CUtensorMap tm_out, const Params p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Ctl &c = *reinterpret_cast<Ctl *>(smem + kCtl);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = p.E;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) { mbar_init(&c.full[s], 1); mbar_init(&c.empty[s], 2); }
        for (int b = 0; b < 4; ++b) { mbar_init(&c.tfull[b >> 1][b & 1], 1); mbar_init(&c.tempty[b >> 1][b & 1], kEpiWarps / 2); }
        for (int h = 0; h < 2; ++h) mbar_init(&c.drain[h], 1);
        if (EXPIRE) mbar_init(&c.never, 1);
        c.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_x)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_w0)) : "memory");
        if (MODE == GATEUP)
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_w1)) : "memory");
    }
    if (warp == 3) tmem_alloc(&c.tmem_base, TMEM_COLS);
    tc_fence_before();
    pdl_enter();
    load_groups(c.g, p);
    __syncthreads();
    if (warp == 0) scan_groups(c.g, p, BM, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    const uint32_t tmem = c.tmem_base;
    const int total = c.g.total, first = blockIdx.x, stride = gridDim.x;
    // (a search and two divides a tile, 500 to 1200 clocks at each tile's end)
    if (threadIdx.x < kTable && first + (int)threadIdx.x * stride < total)
        c.tiles[threadIdx.x] = tile_at(c.g, E, first + threadIdx.x * stride, BM);
    __syncthreads();
    auto nth_tile = [&](int i, int t) { return i < kTable ? c.tiles[i] : tile_at(c.g, E, t, BM); };
    volatile int *abort_flag = &c.abort_flag;
    uint32_t issued = 0;   // blocks this warp has loaded or multiplied
    if (warp < 4) {
        // (inside the branch: the compiler gives each side its own limit)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsAux));
        if (warp == 0) {
            // -------------------------------------------- loads
            uint32_t it = 0;
            bool ok = !(EXPIRE && expires(p, LOADS)) || __all_sync(0xffffffffu, bar_wait(&c.never, 0, abort_flag, p.expire_ns));
            for (int t = first, i = 0; t < total && ok; t += stride, ++i) {
                const Tile tile = nth_tile(i, t);
                const int boxes = (tile.cnt + ABOX - 1) / ABOX;   // only as many as the tile has rows
                for (int kb = 0; kb < p.KB; ++kb, ++it) {
                    const int s = it % STAGES;
                    ok = __all_sync(0xffffffffu, bar_wait(&c.empty[s], ((it / STAGES) & 1u) ^ 1u, abort_flag));
                    if (!ok) break;
                    uint8_t *sa = smem + s * STAGE, *sb = sa + A_BYTES;
                    if (lane == 0) {
                        mbar_expect_tx(&c.full[s], (uint32_t)(boxes * ABOX * BK) + B_BYTES);
                        if (MODE == GATEUP) {
                            // per column half: 64 rows of W_gate, the same 64 of W_up
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint8_t *at = sb + h * (B_BYTES / 2);
                                const int n = tile.nt * (BN / 2) + h * 64;
                                tma_load_3d(at, &tm_w0, &c.full[s], kb * BK, n, tile.e);
                                tma_load_3d(at + B_BYTES / 4, &tm_w1, &c.full[s], kb * BK, n, tile.e);
                            }
                        } else {
                            tma_load_3d(sb, &tm_w0, &c.full[s], kb * BK, tile.nt * BN, tile.e);
                        }
                    }
                    __syncwarp();
                    if (lane < boxes)
                        tma_load_2d(sa + lane * ABOX * BK, &tm_x, &c.full[s], kb * BK, tile.row0 + lane * ABOX);
                }
            }
            if (!ok) {
                if (lane == 0) flag_status(p.status, kDevTimeout);
                c.abort_flag = 1;
            }
            issued = it;
        } else if (warp == 1 || warp == 2) {
            // -------------------------------------------- multiply
            // Warp 1 multiplies the first column half, warp 2 the second, into
            // TMEM buffers of their own: a buffer's turn -- MMAs, their commit,
            // the epilogue's reads, its arrival -- takes several times as long as
            // the MMAs, and four buffers in turn hide more of it than two.  The
            // whole warp runs the loop and one elected lane issues, so that the
            // descriptors stay in uniform registers (a loop of lane 0 alone: 80
            // clocks to issue an MMA).
            constexpr uint32_t idesc = idesc_e4m3(BM, BN / 2);
            const bool leader = elect_one();
            const int h = warp - 1;
            const uint32_t ring = smem_u32(smem), d0 = tmem + h * (BN / 2);
            uint32_t it = 0;
            bool ok = true;
            for (int t = first; t < total && ok; t += stride) {
                for (int kb = 0; kb < p.KB; ++kb, ++it) {
                    const int s = it % STAGES;
                    const uint32_t b = it & 1u;
                    ok = bar_wait(&c.tempty[b][h], ((it >> 1) & 1u) ^ 1u, abort_flag) &&
                         bar_wait(&c.full[s], (it / STAGES) & 1u, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t da = sw128_desc(ring + s * STAGE);
                    const uint64_t db = sw128_desc(ring + s * STAGE + A_BYTES + h * (B_BYTES / 2));
                    if (leader) {
                        umma_f8<false>(d0 + b * BN, da, db, idesc);
#pragma unroll
                        for (int kk = 1; kk < BK / 32; ++kk)
                            umma_f8<true>(d0 + b * BN, desc_step(da, kk * 32), desc_step(db, kk * 32), idesc);
                        umma_commit(&c.tfull[b][h]);
                        umma_commit(&c.empty[s]);
                    }
                }
            }
            if (!ok) {
                if (leader) flag_status(p.status, kDevTimeout);
                c.abort_flag = 1;
            }
            issued = it;
        }
    } else {
        // ------------------------------------------------ sums and output
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const int row = quarter * 32 + lane;
        uint8_t *stg = smem + kRing + (warp - 4) * kStaging;
        uint32_t it = 0;
        // (once false, no more waits: the remaining rows become NaN)
        bool ok = !(EXPIRE && expires(p, SUMS)) || __all_sync(0xffffffffu, bar_wait(&c.never, 0, abort_flag, p.expire_ns));
        Tile next;
        const float *xs = nullptr;
        uint32_t ws = 0;   // place of the weight scales (one for each 16 KB of codes: 32 bits do)
        float nx = 0.f, n0 = 0.f, n1 = 0.f;   // the next block's scales
        // tile t's place and its first scales, asked for ahead of the tile before's output
        auto enter = [&](int i, int t) {
            if (t >= total) return;
            next = nth_tile(i, t);
            xs = row < next.cnt ? p.x_s + (long long)(next.row0 + row) * p.KB : nullptr;
            // the weight scales of the columns this warp sums: gate and up, or
            // one 128-column block (none past the last: its sums are zero)
            const int nb = MODE == GATEUP ? next.nt : min(next.nt * 2 + half, p.NB - 1);
            ws = (uint32_t)((next.e * p.NB + nb) * p.KB);
            nx = xs ? __ldg(xs) : 0.f;
            n0 = __ldg(p.w_s[0] + ws);
            if (MODE == GATEUP) n1 = __ldg(p.w_s[1] + ws);
        };
        enter(0, first);
        for (int t = first, n = 1; t < total; t += stride, ++n) {
            const Tile tile = next;
            const bool valid = row < tile.cnt;
            const long long r = tile.row0 + row;
            uint64_t acc[64];   // 128 sums: PRODUCT columns half*128 ..; GATEUP 64 of gate, 64 of up
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0ull;
#pragma unroll 1
            for (int kb = 0; kb < p.KB; ++kb, ++it) {
                const uint32_t b = it & 1u;
                const float f0 = nx * n0, f1 = MODE == GATEUP ? nx * n1 : f0;
                const uint64_t m0 = pack2(__float_as_uint(f0), __float_as_uint(f0));
                const uint64_t m1 = pack2(__float_as_uint(f1), __float_as_uint(f1));
                if (kb + 1 < p.KB) {
                    nx = xs ? __ldg(xs + kb + 1) : 0.f;
                    n0 = __ldg(p.w_s[0] + ++ws);
                    if (MODE == GATEUP) n1 = __ldg(p.w_s[1] + ws);
                }
                ok = ok && __all_sync(0xffffffffu, bar_wait(&c.tfull[b][half], (it >> 1) & 1u, abort_flag));
                if (!ok) continue;   // (TMEM that no MMA has written is not read)
                tc_fence_after();
                const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16) + b * BN + half * (BN / 2);
                // Two loads of 64 columns: the buffer's reads are in the chain that
                // decides how soon it can be filled again (eight loads of 16, one
                // ahead of the sums, took 540 clocks of a block's 900).
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t v[64];
                    tmem_ld64_wait(base + j * 64, v);
                    if (j == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&c.tempty[b][half]);
                    }
                    const uint64_t m = j ? m1 : m0;
#pragma unroll
                    for (int i = 0; i < 32; ++i) fma2(acc[j * 32 + i], pack2(v[2 * i], v[2 * i + 1]), m);
                }
            }
            enter(n, t + stride);
            if (!ok) {
                // (the other roles may have left their loops: this warp reports too)
                if (lane == 0) flag_status(p.status, kDevTimeout);
                c.abort_flag = 1;
                const uint64_t nan2 = 0x7fffffff7fffffffull;
#pragma unroll
                for (int i = 0; i < 64; ++i) acc[i] = nan2;
            }
            auto val = [&](int i) { return (i & 1) ? hi2(acc[i >> 1]) : lo2(acc[i >> 1]); };
            if constexpr (MODE == GATEUP) {
                uint32_t m = 0u;
                float h[64];
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    h[i] = swiglu(val(i), val(64 + i));
                    m = max(m, mag_bits(h[i]));
                }
                // the other half of the row's 128 channels is in the warp of the
                // same quarter: the two meet at a barrier of their own (both
                // take every turn of the tile loop, whatever happened before)
                c.amax[half][row] = m;
                asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
                m = max(m, c.amax[half ^ 1][row]);
                asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
                const float s = block_scale(m), f = code_factor(s);
                const int c0 = tile.nt * (BN / 2) + half * 64;
                uint4 d[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float *v = h + 16 * i;
                    d[i] = make_uint4(encode4(v[0], v[1], v[2], v[3], f), encode4(v[4], v[5], v[6], v[7], f),
                                      encode4(v[8], v[9], v[10], v[11], f), encode4(v[12], v[13], v[14], v[15], f));
                }
                store_rows(stg, lane, d, p.h_q + (r - lane) * p.N + c0, p.N, tile.cnt - quarter * 32, p.N - c0, 1);
                if (valid && half == 0) p.h_s[r * p.NB + tile.nt] = s;
            } else {
                const int c0 = tile.nt * BN + half * (BN / 2), rows = tile.cnt - quarter * 32;
                const bool f32 = p.out_f32;
                const int size = f32 ? 4 : 2;
                // Slices with all of their 32 rows go out by TMA: the warp goes on
                // to the next tile while they drain.  (All CTAs end their tiles
                // together, and waiting for the burst of their stores to be taken
                // cost 2 us a tile.)
                const bool tma = p.out_tma && rows >= 32;
                if (lane == 0) bulk_wait_read();   // the staging of the tile before has been read
                __syncwarp();
                // the k-th 128 bytes of each row: 64 columns of bf16, 32 of fp32
                auto piece = [&](int k, uint4 (&d)[8]) {
                    if (f32) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const int i = k * 32 + q * 4;
                            d[q] = make_uint4(__float_as_uint(val(i)), __float_as_uint(val(i + 1)),
                                              __float_as_uint(val(i + 2)), __float_as_uint(val(i + 3)));
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const int i = (k & 1) * 64 + q * 8;
                            d[q] = make_uint4(bf16x2(val(i), val(i + 1)), bf16x2(val(i + 2), val(i + 3)),
                                              bf16x2(val(i + 4), val(i + 5)), bf16x2(val(i + 6), val(i + 7)));
                        }
                    }
                };
                const int cols = 128 / size;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (!f32 && k >= 2) break;
                    const int n = c0 + k * cols;
                    uint8_t *at = stg + (k & 1) * 4096;
                    uint4 d[8];
                    piece(k, d);
                    if (tma) {
                        if (k == 2) {   // the first pieces' staging again
                            if (lane == 0) bulk_wait_read();
                            __syncwarp();
                        }
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            *reinterpret_cast<uint4 *>(at + lane * 128 + ((q ^ (lane & 7)) << 4)) = d[q];
                        if (k & 1) {
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                if (n - cols < p.N) tma_store_2d(&tm_out, stg, n - cols, (int)r);
                                if (n < p.N) tma_store_2d(&tm_out, at, n, (int)r);
                                bulk_commit();
                            }
                        }
                    } else if (p.out_vec) {
                        uint8_t *g = static_cast<uint8_t *>(p.out) + ((r - lane) * p.ldo + n) * size;
                        const int bytes = (p.N - n) * size;
                        const uint4 lo[4] = {d[0], d[1], d[2], d[3]}, hi[4] = {d[4], d[5], d[6], d[7]};
                        store_rows(at, lane, lo, g, p.ldo * size, rows, bytes, size);
                        store_rows(at, lane, hi, g + 64, p.ldo * size, rows, bytes - 64, size);
                    } else {
                        // rows that are not 16-byte aligned: staged as for TMA, then a
                        // row at a time, 32 neighbouring elements an instruction
                        __syncwarp();
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            *reinterpret_cast<uint4 *>(at + lane * 128 + ((q ^ (lane & 7)) << 4)) = d[q];
                        __syncwarp();
                        if (f32) store_elements<uint32_t>(p, at, lane, r - lane, n, min(rows, 32));
                        else store_elements<uint16_t>(p, at, lane, r - lane, n, min(rows, 32));
                    }
                }
            }
        }
        if (MODE == PRODUCT && lane == 0) bulk_wait_all();
    }

    __syncthreads();
    if (*abort_flag) {
        // A role gave up, and nothing says that the sums' warps have waited for
        // what the others issued (which may have left their loops before): loads
        // land before the CTA exits, MMAs end before TMEM is freed.
        volatile int no_abort = 0;
        if (warp == 0) {
            for (uint32_t j = issued >= STAGES ? issued - STAGES : 0; j < issued; ++j)
                bar_wait(&c.full[j % STAGES], (j / STAGES) & 1u, &no_abort, 1000000ull);
        } else if ((warp == 1 || warp == 2) && issued > 0) {
            if (elect_one()) umma_commit(&c.drain[warp - 1]);
            bar_wait(&c.drain[warp - 1], 0, &no_abort);
        }
        __syncthreads();
    }
    if (warp == 3) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Rows gathered through perm_tok into group order, codes and scales, a warp to
// a row; an index outside [0, x_rows) gives a row of zeros.
constexpr int kGatherWarps = 8;
__global__ void __launch_bounds__(32 * kGatherWarps)
gather_kernel(const uint8_t *__restrict__ x_q, const float *__restrict__ x_s, long long ldx, int x_rows, int K, int KB,
              const int32_t *__restrict__ perm_tok, int rows, uint8_t *__restrict__ g_q, float *__restrict__ g_s)
{
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const long long r = (long long)blockIdx.x * kGatherWarps + (threadIdx.x >> 5);
    if (r >= rows) return;
    const int tok = __ldg(perm_tok + r);
    const bool in = tok >= 0 && tok < x_rows;
    const uint4 *src = reinterpret_cast<const uint4 *>(x_q + (in ? tok : 0) * ldx);
    uint4 *dst = reinterpret_cast<uint4 *>(g_q + r * K);
    constexpr int U = 4;   // loads in flight per lane
    for (int i0 = lane; i0 < K / 16; i0 += 32 * U) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[u] = in && i0 + 32 * u < K / 16 ? __ldg(src + i0 + 32 * u) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + 32 * u < K / 16) dst[i0 + 32 * u] = v[u];
    }
    for (int i = lane; i < KB; i += 32) g_s[r * KB + i] = in ? __ldg(x_s + (long long)tok * KB + i) : 0.f;
}

// ------------------------------------------------------------------- host
size_t gathered_codes_bytes(int rows, int K) { return align_up((size_t)rows * K, 256); }

// out [rows, N], rows ldo apart, box {128 bytes of columns, 32 rows}, 128-byte swizzle
bool out_map(CUtensorMap *m, const Params &p)
{
    auto enc = tc::encode_fn();
    if (!enc) return false;
    const int size = p.out_f32 ? 4 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)p.N, (cuuint64_t)p.rows};
    const cuuint64_t strides[1] = {(cuuint64_t)p.ldo * size};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / size), 32};
    const cuuint32_t one[2] = {1, 1};
    return enc(m, p.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.out, dims, strides,
               box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, bool EXPIRE>
cudaError_t launch_kernel(const CUtensorMap &x, const CUtensorMap &w0, const CUtensorMap &w1, const CUtensorMap &out,
                          const Params &p, long long tiles, int num_sms, cudaStream_t stream)
{
    static PerDeviceFlag done;
    const int dev = current_device();
    auto *kern = product_kernel<MODE, EXPIRE>;
    if (!done.done(dev)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e != cudaSuccess) return e;
        done.mark(dev);
    }
    return launch_pdl(kern, dim3((unsigned)(tiles < num_sms ? tiles : num_sms)), dim3(kThreads), kSmem, stream, x, w0,
                      w1, out, p);
}

template <int MODE>
cudaError_t launch_product(const void *x_q, long long ldx, const void *w0, const void *w1, Params p, void *workspace,
                           cudaStream_t stream)
{
    const int num_sms = device_sm_count();
    if (decode_fits(p, num_sms)) return launch_decode<MODE>(x_q, ldx, w0, w1, p, num_sms, stream);
    if (p.perm_tok) {
        // Rows go into group order once, ahead of the product: every column
        // tile would gather them again, and a loop that copies rows feeds the
        // tensor cores more slowly than TMA does (4096 rows x 2048 against 2 x
        // 2816 columns of 16 experts: 100 us gathering in the kernel, 62 us on
        // rows in order, plus 4 us for this copy).
        uint8_t *g_q = static_cast<uint8_t *>(workspace);
        float *g_s = reinterpret_cast<float *>(g_q + gathered_codes_bytes(p.rows, p.K));
        const cudaError_t e = launch_pdl(gather_kernel, dim3((unsigned)ceil_div(p.rows, kGatherWarps)),
                                         dim3(32 * kGatherWarps), 0, stream, static_cast<const uint8_t *>(x_q), p.x_s,
                                         ldx, p.x_rows, p.K, p.KB, p.perm_tok, p.rows, g_q, g_s);
        if (e != cudaSuccess) return e;
        x_q = g_q;
        ldx = p.K;
        p.x_s = g_s;
        p.x_rows = p.rows;
        p.perm_tok = nullptr;
    }
    p.n_tiles = ceil_div(p.N, MODE == GATEUP ? BN / 2 : BN);
    // most tiles there can be: an expert with r rows has (r - 1) / BM + 1, so as
    // many experts as possible with rows, and the rest of the rows in whole tiles
    const long long experts = p.E < p.rows ? p.E : p.rows;
    const long long tiles = ((p.rows - experts) / BM + experts) * p.n_tiles;
    if (tiles > 0x3fffffffLL) return cudaErrorInvalidValue;
    CUtensorMap mx, mw0, mw1, mout;
    constexpr uint32_t wbox = MODE == GATEUP ? BN / 4 : BN;
    if (!code_map(&mx, x_q, 0, p.x_rows, p.K, ldx, ABOX) || !code_map(&mw0, w0, p.E, p.N, p.K, p.K, wbox))
        return cudaErrorInvalidValue;
    if (MODE != GATEUP) mw1 = mw0;
    else if (!code_map(&mw1, w1, p.E, p.N, p.K, p.K, wbox)) return cudaErrorInvalidValue;
    // the output as a tensor, where its rows suit TMA: it stores whole 16-byte
    // parts, the last one of a row too, so rows that end inside one would lose
    // what lies behind them (another column slice of the caller's tensor)
    p.out_tma = MODE == PRODUCT && p.out_vec && p.N % (p.out_f32 ? 4 : 8) == 0;
    if (!p.out_tma) mout = mx;
    else if (!out_map(&mout, p)) return cudaErrorInvalidValue;
    if (p.expire_ns) return launch_kernel<MODE, true>(mx, mw0, mw1, mout, p, tiles, num_sms, stream);
    return launch_kernel<MODE, false>(mx, mw0, mw1, mout, p, tiles, num_sms, stream);
}

bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The checks the products share; MOE_OK with *go = false for an empty call.
moe_status product_args(const void *x_q, const float *x_s, int x_rows, int K, long long ldx, const void *w_q,
                        const float *w_s, int E, int N, const int32_t *offsets, const int32_t *perm_tok, int rows,
                        const void *status, const void *workspace, size_t ws_bytes, bool *go)
{
    *go = false;
    if (x_rows < 0 || rows < 0 || K <= 0 || K % 16 || N <= 0 || E <= 0) return MOE_ERR_INVALID_ARG;
    if (ldx < K || ldx % 16) return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts) return MOE_ERR_UNSUPPORTED;
    if (E > 1 && !offsets && rows > 0) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!perm_tok && rows > x_rows) return MOE_ERR_INVALID_ARG;
    if (x_rows == 0) return MOE_ERR_INVALID_ARG;
    if (rows > INT32_MAX / 2 || x_rows > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
    if (!x_q || !x_s || !w_q || !w_s) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(x_q, 16) || !aligned_to(w_q, 16) || !aligned_to(x_s, 4) || !aligned_to(w_s, 4) ||
        !aligned_to(offsets, 4) || !aligned_to(perm_tok, 4) || !aligned_to(status, 4))
        return MOE_ERR_INVALID_ARG;
    if (perm_tok) {
        if (!workspace || !aligned_to(workspace, 256)) return MOE_ERR_INVALID_ARG;
        if (ws_bytes < moe_fp8b_workspace_size(rows, K)) return MOE_ERR_WORKSPACE;
    }
    *go = true;
    return MOE_OK;
}

Params params_of(const float *x_s, int x_rows, int K, const float *s0, const float *s1, int E, int N,
                 const int32_t *offsets, const int32_t *perm_tok, int rows, uint32_t *status)
{
    Params p{};
    p.x_s = x_s; p.w_s[0] = s0; p.w_s[1] = s1; p.offsets = offsets; p.perm_tok = perm_tok;
    p.E = E; p.rows = rows; p.x_rows = x_rows; p.K = K; p.N = N;
    p.KB = ceil_div(K, kBlock); p.NB = ceil_div(N, kBlock);
    p.status = status;
    return p;
}

}  // namespace fp8b
}  // namespace moe

using namespace moe;
using namespace moe::fp8b;

namespace {

bool hook_limit_ok(uint32_t wait_ns) { return wait_ns > 0 && wait_ns <= 100000000u; }

moe_status grouped_gemm(const void *x_q, const float *x_s, int x_rows, int K, long long ldx, const void *w_q,
                        const float *w_s, int E, int N, const int32_t *offsets, const int32_t *perm_tok, int rows,
                        void *out, moe_dtype out_dt, long long ldo, void *workspace, size_t ws_bytes, uint32_t *status,
                        uint32_t expire_ns, Role expire_role, moe_stream stream)
{
    bool go;
    const moe_status st = product_args(x_q, x_s, x_rows, K, ldx, w_q, w_s, E, N, offsets, perm_tok, rows, status,
                                        workspace, ws_bytes, &go);
    if (st != MOE_OK) return st;
    if ((out_dt != MOE_F32 && out_dt != MOE_BF16) || ldo < N) return MOE_ERR_INVALID_ARG;
    if (!go) return MOE_OK;
    if (!out || !aligned_to(out, out_dt == MOE_F32 ? 4 : 2)) return MOE_ERR_INVALID_ARG;
    Params p = params_of(x_s, x_rows, K, w_s, nullptr, E, N, offsets, perm_tok, rows, status);
    p.expire_ns = expire_ns;
    p.expire_role = expire_role;
    p.out = out; p.ldo = ldo; p.out_f32 = out_dt == MOE_F32;
    p.out_vec = ldo % (out_dt == MOE_F32 ? 4 : 8) == 0 && aligned_to(out, 16);
    const cudaError_t e = launch_product<PRODUCT>(x_q, ldx, w_q, nullptr, p, workspace, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status gate_up(const void *x_q, const float *x_s, int x_rows, int d, long long ldx, const void *wg_q,
                   const float *wg_s, const void *wu_q, const float *wu_s, int E, int F, const int32_t *offsets,
                   const int32_t *perm_tok, int rows, void *h_q, float *h_s, void *workspace, size_t ws_bytes,
                   uint32_t *status, uint32_t expire_ns, Role expire_role, moe_stream stream)
{
    bool go;
    const moe_status st = product_args(x_q, x_s, x_rows, d, ldx, wg_q, wg_s, E, F, offsets, perm_tok, rows, status,
                                        workspace, ws_bytes, &go);
    if (st != MOE_OK) return st;
    if (F % 16) return MOE_ERR_INVALID_ARG;
    if (!go) return MOE_OK;
    if (!wu_q || !wu_s || !h_q || !h_s) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(wu_q, 16) || !aligned_to(wu_s, 4) || !aligned_to(h_q, 16) || !aligned_to(h_s, 4))
        return MOE_ERR_INVALID_ARG;
    Params p = params_of(x_s, x_rows, d, wg_s, wu_s, E, F, offsets, perm_tok, rows, status);
    p.expire_ns = expire_ns;
    p.expire_role = expire_role;
    p.h_q = static_cast<uint8_t *>(h_q); p.h_s = h_s;
    const cudaError_t e = launch_product<GATEUP>(x_q, ldx, wg_q, wu_q, p, workspace, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t moe_fp8b_workspace_size(int rows, int K)
{
    if (rows < 0 || K <= 0 || K % 16) return 0;
    return gathered_codes_bytes(rows, K) + align_up((size_t)rows * ceil_div(K, kBlock) * 4, 256);
}

moe_status moe_grouped_gemm_fp8b(const void *x_q, const float *x_s, int x_rows, int K, long long ldx,
                                 const void *w_q, const float *w_s, int E, int N, const int32_t *offsets,
                                 const int32_t *perm_tok, int rows, void *out, moe_dtype out_dt, long long ldo,
                                 void *workspace, size_t ws_bytes, uint32_t *status, moe_stream stream)
{
    return grouped_gemm(x_q, x_s, x_rows, K, ldx, w_q, w_s, E, N, offsets, perm_tok, rows, out, out_dt, ldo, workspace,
                        ws_bytes, status, 0, LOADS, stream);
}

moe_status moe_grouped_gemm_fp8b_expire_wait(const void *x_q, const float *x_s, int x_rows, int K, long long ldx,
                                             const void *w_q, const float *w_s, int E, int N, const int32_t *offsets,
                                             const int32_t *perm_tok, int rows, void *out, moe_dtype out_dt,
                                             long long ldo, void *workspace, size_t ws_bytes, uint32_t *status,
                                             uint32_t wait_ns, moe_stream stream)
{
    if (!hook_limit_ok(wait_ns)) return MOE_ERR_INVALID_ARG;
    return grouped_gemm(x_q, x_s, x_rows, K, ldx, w_q, w_s, E, N, offsets, perm_tok, rows, out, out_dt, ldo, workspace,
                        ws_bytes, status, wait_ns, LOADS, stream);
}

moe_status moe_grouped_gemm_fp8b_expire_sums(const void *x_q, const float *x_s, int x_rows, int K, long long ldx,
                                             const void *w_q, const float *w_s, int E, int N, const int32_t *offsets,
                                             const int32_t *perm_tok, int rows, void *out, moe_dtype out_dt,
                                             long long ldo, void *workspace, size_t ws_bytes, uint32_t *status,
                                             uint32_t wait_ns, moe_stream stream)
{
    if (!hook_limit_ok(wait_ns)) return MOE_ERR_INVALID_ARG;
    return grouped_gemm(x_q, x_s, x_rows, K, ldx, w_q, w_s, E, N, offsets, perm_tok, rows, out, out_dt, ldo, workspace,
                        ws_bytes, status, wait_ns, SUMS, stream);
}

moe_status moe_gemm_fp8b(const void *x_q, const float *x_s, int T, int K, long long ldx, const void *w_q,
                         const float *w_s, int N, void *out, moe_dtype out_dt, long long ldo, uint32_t *status,
                         moe_stream stream)
{
    return moe_grouped_gemm_fp8b(x_q, x_s, T, K, ldx, w_q, w_s, 1, N, nullptr, nullptr, T, out, out_dt, ldo, nullptr, 0,
                                 status, stream);
}

moe_status moe_gate_up_fp8b(const void *x_q, const float *x_s, int x_rows, int d, long long ldx, const void *wg_q,
                            const float *wg_s, const void *wu_q, const float *wu_s, int E, int F,
                            const int32_t *offsets, const int32_t *perm_tok, int rows, void *h_q, float *h_s,
                            void *workspace, size_t ws_bytes, uint32_t *status, moe_stream stream)
{
    return gate_up(x_q, x_s, x_rows, d, ldx, wg_q, wg_s, wu_q, wu_s, E, F, offsets, perm_tok, rows, h_q, h_s, workspace,
                   ws_bytes, status, 0, LOADS, stream);
}

moe_status moe_gate_up_fp8b_expire_wait(const void *x_q, const float *x_s, int x_rows, int d, long long ldx,
                                        const void *wg_q, const float *wg_s, const void *wu_q, const float *wu_s, int E,
                                        int F, const int32_t *offsets, const int32_t *perm_tok, int rows, void *h_q,
                                        float *h_s, void *workspace, size_t ws_bytes, uint32_t *status,
                                        uint32_t wait_ns, moe_stream stream)
{
    if (!hook_limit_ok(wait_ns)) return MOE_ERR_INVALID_ARG;
    return gate_up(x_q, x_s, x_rows, d, ldx, wg_q, wg_s, wu_q, wu_s, E, F, offsets, perm_tok, rows, h_q, h_s, workspace,
                   ws_bytes, status, wait_ns, LOADS, stream);
}

moe_status moe_gate_up_fp8b_expire_sums(const void *x_q, const float *x_s, int x_rows, int d, long long ldx,
                                        const void *wg_q, const float *wg_s, const void *wu_q, const float *wu_s, int E,
                                        int F, const int32_t *offsets, const int32_t *perm_tok, int rows, void *h_q,
                                        float *h_s, void *workspace, size_t ws_bytes, uint32_t *status,
                                        uint32_t wait_ns, moe_stream stream)
{
    if (!hook_limit_ok(wait_ns)) return MOE_ERR_INVALID_ARG;
    return gate_up(x_q, x_s, x_rows, d, ldx, wg_q, wg_s, wu_q, wu_s, E, F, offsets, perm_tok, rows, h_q, h_s, workspace,
                   ws_bytes, status, wait_ns, SUMS, stream);
}

}  // extern "C"
