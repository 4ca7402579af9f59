// i8_quant.cu -- int8 codes of rows, one fp32 scale per row:
//   s = max|x| / 127,   c = the whole number nearest to 127 x / max|x|, ties to even.
//
// The codes are those of the quotient itself, not of a rounded one: 127 / max|x| is
// held in two fp32 numbers (a quotient and the quotient of its remainder, Dekker 1971),
// so x times their sum is off by half a unit in the last place and little more.  A
// bf16 quotient that is not a tie is at least 2^-17 of itself away from one (127 x and
// max|x| have short significands), so its rounding cannot reach it, and a tie is exact;
// an fp32 quotient that comes out within 2^-15 of a tie is compared with it in 64
// bits, where both sides are exact (31 and 32 bits).
//
// What bounds it: memory.  Every value is read once into registers and stays there
// between the maximum and the codes.  8192 x 2816 in bf16 take 11.8 us (5.9 TB/s, 88 % of the
// measured copy rate), in fp32 20.9 (83 %); one row of 2048 1.5, a kernel's start and end.
#include <type_traits>

#include "i8.h"

namespace moe {
namespace i8 {

constexpr float kCodeMax = 127.0f;
constexpr float kLeastTop = 0x1.fcp-120f;        // 127 * 2^-126: below, top / 127 rounds to less than 2^-126
constexpr uint32_t kInfBits = 0x7f800000u;
constexpr int kQuantThreads = 512;              // most of a CTA

// |v| as bits: their order is that of the magnitudes, infinity above every finite
// value and NaN above infinity, so a maximum does not lose a NaN.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Eight values as loaded.
template <typename XT> struct Raw8;
template <> struct Raw8<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = __ldg(reinterpret_cast<const uint4 *>(p));
        b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ float get(int i) const
    {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        return __uint_as_float(w[i]);
    }
    __device__ __forceinline__ uint32_t max_bits() const
    {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, mag_bits(get(i)));
        return m;
    }
};
template <> struct Raw8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ float get(int i) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
        return (i & 1) ? bf16hi(w[i >> 1]) : bf16lo(w[i >> 1]);
    }
    __device__ __forceinline__ uint32_t max_bits() const
    {
        const uint32_t k = 0x7fff7fffu;
        const uint32_t m = __vmaxu2(__vmaxu2(a.x & k, a.y & k), __vmaxu2(a.z & k, a.w & k));
        return max(m << 16, m & 0xffff0000u);
    }
};

// What takes a row's values to codes.
struct Factor {
    float hi, lo, top;   // 127 / max|x| = hi + lo; zeros for a row of zero codes
};
__device__ __forceinline__ Factor factor_of(uint32_t top_bits)
{
    const float top = __uint_as_float(top_bits);
    Factor f{0.f, 0.f, top};
    if (top_bits < kInfBits && top >= kLeastTop) {   // (so that 127 / max|x| is finite)
        f.hi = kCodeMax / top;
        // the remainder's quotient, to 2^-22 of itself: 1 / top is hi / 127
        f.lo = fmaf(-f.hi, top, kCodeMax) * (f.hi * (1.0f / kCodeMax));
    }
    return f;
}
__device__ __forceinline__ float scale_of(uint32_t top_bits)
{
    const float top = __uint_as_float(top_bits);
    if (top_bits >= kInfBits) return __uint_as_float(0x7fffffffu);   // an infinity or a NaN: NaN scale, zero codes
    return top < kLeastTop ? 0.f : top / kCodeMax;
}
// Adding 1.5 * 2^23 leaves the nearest whole number in the low bits, ties to even (a
// conversion to int runs at a quarter of the rate).  A value of NaN or beyond the range comes
// only with a row of zero codes.
constexpr float kWhole = 12582912.0f;
__device__ __forceinline__ uint64_t pack2(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
// Two values' codes in the low bytes (two fp32 operations an instruction, each rounded as
// alone).
__device__ __forceinline__ void codes2(float x0, float x1, const Factor &f, uint32_t &c0, uint32_t &c1)
{
    const uint64_t x = pack2(x0, x1);
    uint64_t t;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(x), "l"(pack2(f.lo, f.lo)));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(t) : "l"(x), "l"(pack2(f.hi, f.hi)));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(t) : "l"(pack2(kWhole, kWhole)));
    c0 = (uint32_t)t;
    c1 = (uint32_t)(t >> 32);
}
// One fp32 value's code: near a tie, by both sides in 64 bits.
__device__ __forceinline__ uint32_t code_of(float x, const Factor &f)
{
    const float q = fmaf(x, f.hi, x * f.lo), t = q + kWhole;
    uint32_t c = __float_as_uint(t);
    if (fabsf(q - (t - kWhole)) > 0.5f - 0x1p-15f) {
        const float low = floorf(fabsf(q));
        const double left = 127.0 * (double)fabsf(x), right = ((double)low + 0.5) * (double)f.top;
        const int l = (int)low, n = left > right ? l + 1 : left < right ? l : l + (l & 1);
        c = (uint32_t)(x < 0.f ? -n : n);
    }
    return c;
}
template <typename XT> __device__ __forceinline__ uint2 codes_of(const Raw8<XT> &r, const Factor &f)
{
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t c[4];
        if constexpr (std::is_same<XT, float>::value) {
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = code_of(r.get(4 * h + i), f);
        } else {
            codes2(r.get(4 * h), r.get(4 * h + 1), f, c[0], c[1]);
            codes2(r.get(4 * h + 2), r.get(4 * h + 3), f, c[2], c[3]);
        }
        w[h] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    }
    // (zero codes, whatever the products of a row's infinities and NaN with 0 are)
    return f.hi == 0.f ? make_uint2(0u, 0u) : make_uint2(w[0], w[1]);
}

// blockDim.x threads (a multiple of 32) to a row, NV chunks of 8 values each, all in
// registers; rows wider than that (LONG) are read a second time.
template <typename XT, int NV, bool LONG>
__global__ void __launch_bounds__(kQuantThreads)
quant_rows_kernel(const XT *__restrict__ x, long long rows, int cols, long long ldx,
                  uint8_t *__restrict__ codes, float *__restrict__ scales)
{
    pdl_enter();
    __shared__ uint32_t part[kQuantThreads / 32];
    const int lanes = blockDim.x, lane = threadIdx.x;
    const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    const int chunks = cols / 8;
    Raw8<XT> r[NV];
    uint32_t m = 0u;
    if (row < rows) {
        const XT *p = x + row * ldx;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = lane + i * lanes;
            if (c < chunks) r[i].load(p + c * 8);
            else r[i].zero();
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) m = max(m, r[i].max_bits());
        if (LONG) {
            for (int c = lane + NV * lanes; c < chunks; c += lanes) {
                Raw8<XT> v;
                v.load(p + (long long)c * 8);
                m = max(m, v.max_bits());
            }
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lanes > 32) {   // (uniform over the CTA)
        const int n = lanes >> 5, l = lane & 31;
        uint32_t *mine = part + threadIdx.y * n;
        if (l == 0) mine[lane >> 5] = m;
        __syncthreads();
        m = __reduce_max_sync(0xffffffffu, l < n ? mine[l] : 0u);
    }
    if (row >= rows) return;
    const Factor f = factor_of(m);
    uint8_t *o = codes + row * cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = lane + i * lanes;
        if (c < chunks) *reinterpret_cast<uint2 *>(o + c * 8) = codes_of<XT>(r[i], f);
    }
    if (LONG) {
        const XT *p = x + row * ldx;
        for (int c = lane + NV * lanes; c < chunks; c += lanes) {
            Raw8<XT> v;
            v.load(p + (long long)c * 8);
            *reinterpret_cast<uint2 *>(o + (long long)c * 8) = codes_of<XT>(v, f);
        }
    }
    if (lane == 0) scales[row] = scale_of(m);
}

template <typename XT>
cudaError_t launch_quant(const void *x, int rows, int cols, long long ldx, uint8_t *codes, float *scales, cudaStream_t s)
{
    constexpr int kMost = sizeof(XT) == 4 ? 4 : 8;   // chunks a thread holds: 32 registers
    const int chunks = cols / 8;
    // Many rows: as few threads to a row as hold it with most of their chunks in use (a
    // warp needs no barrier, and several chunks are in flight a thread); few rows: as many
    // threads as chunks, as they are latency.  (8192 x 2816 in bf16: 64 threads of 8 chunks,
    // of which 352 of 512 are used, 13.5 us; 96 of 4 13.1.)
    int lanes = chunks;
    if (rows >= 16 * device_sm_count()) {
        int best = 0;   // slots that a choice leaves unused, of 1024 for each it has
        for (int nv = kMost; nv >= 1; nv /= 2) {
            const int l = (int)align_up((size_t)ceil_div(chunks, nv), 32), waste = (l * nv - chunks) * 1024 / (l * nv);
            if (nv == kMost || waste < best - 100) { lanes = l; best = waste; }
        }
    }
    lanes = (int)align_up((size_t)(lanes < kQuantThreads ? lanes : kQuantThreads), 32);
    const int nv = ceil_div(chunks, lanes), per = lanes < 128 ? 128 / lanes : 1;
    auto go = [&](auto kern) {
        return launch_pdl(kern, dim3((unsigned)(((long long)rows + per - 1) / per)), dim3(lanes, per), 0, s,
                          static_cast<const XT *>(x), (long long)rows, cols, ldx, codes, scales);
    };
    if (nv <= 1) return go(quant_rows_kernel<XT, 1, false>);
    if (nv <= 2) return go(quant_rows_kernel<XT, 2, false>);
    if (nv <= 4) return go(quant_rows_kernel<XT, 4, false>);
    if (nv <= kMost) return go(quant_rows_kernel<XT, kMost, false>);
    return go(quant_rows_kernel<XT, kMost, true>);
}

}  // namespace i8
}  // namespace moe

using namespace moe;
using namespace moe::i8;

extern "C" moe_status moe_quant_i8(const void *x, moe_dtype x_dt, int rows, int cols, long long ldx, int8_t *codes,
                                   float *scales, moe_stream stream)
{
    auto aligned = [](const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
    if (rows < 0 || cols <= 0 || cols % 16 || (x_dt != MOE_F32 && x_dt != MOE_BF16)) return MOE_ERR_INVALID_ARG;
    if (ldx < cols || ldx % 8) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!x || !codes || !scales || !aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t *q = reinterpret_cast<uint8_t *>(codes);
    const cudaError_t e = x_dt == MOE_F32 ? launch_quant<float>(x, rows, cols, ldx, q, scales, s)
                                          : launch_quant<__nv_bfloat16>(x, rows, cols, ldx, q, scales, s);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
