// quantize.cu -- 8-bit (e4m3) codes with one fp32 step per block of 1 x 128 or
// 128 x 128 values:
//   s_b = fp32(max |x_b| / 448), 1 if that is zero;
//   q = e4m3_nearest_even(clamp(fp32(x / s_b), -448, 448)).
// The quotient is the correctly rounded fp32 one, as for the solver's grid, so
// the codes are a function of the input alone.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "mm.cuh"

namespace bakron {
namespace mm {

namespace {

// Sixteen consecutive values of a row, as loaded.
template <typename T>
struct alignas(32) Run {
    uint32_t w[16 * sizeof(T) / 4];
};

__device__ __forceinline__ void load32(const void *p, uint32_t *v)
{
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
}

// From column c on, zeros from column `cols` on; `align`: bytes that the row's
// start is aligned to (32, 16 or less).
template <typename T>
__device__ __forceinline__ Run<T> load_run(const T *row, int c, int cols, int align)
{
    constexpr int kWords = sizeof(Run<T>::w) / 4;
    Run<T> v;
    if (align >= 32 && c + 16 <= cols) {
#pragma unroll
        for (int i = 0; i < kWords; i += 8) load32((const uint32_t *)(row + c) + i, v.w + i);
    } else if (align >= 16 && c + 16 <= cols) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) *(uint4 *)(v.w + i) = __ldg((const uint4 *)((const uint32_t *)(row + c) + i));
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v.w[i] = c + i < cols ? __float_as_uint(row[c + i]) : 0u;
    } else {
        const uint16_t *h = (const uint16_t *)row;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t lo = c + 2 * i < cols ? h[c + 2 * i] : 0u, hi = c + 2 * i + 1 < cols ? h[c + 2 * i + 1] : 0u;
            v.w[i] = lo | (hi << 16);
        }
    }
    return v;
}
__device__ __forceinline__ int row_align(const void *row)
{
    return ((uintptr_t)row & 31) == 0 ? 32 : ((uintptr_t)row & 15) == 0 ? 16 : 1;
}

// The two numbers of word i of a 16-bit run.
__device__ __forceinline__ float2 pair_of(const Run<__nv_bfloat16> &e, int i)
{
    return make_float2(__uint_as_float(e.w[i] << 16), __uint_as_float(e.w[i] & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_of(const Run<__half> &e, int i) { return __half22float2(*(const __half2 *)&e.w[i]); }
__device__ __forceinline__ float2 pair_of(const Run<float> &e, int i)
{
    return make_float2(__uint_as_float(e.w[2 * i]), __uint_as_float(e.w[2 * i + 1]));
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t m;
    asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
}

// The largest magnitude of the values and `most`, as the bits of the type
// with the sign cleared: ordered like the magnitudes, infinities and NaN above
// every finite value.  16-bit types keep two maxima in one word.
template <typename T>
__device__ __forceinline__ uint32_t most_of(const Run<T> &e, uint32_t most)
{
#pragma unroll
    for (int i = 0; i < (int)sizeof(e.w) / 4; ++i)
        most = sizeof(T) == 4 ? max(most, e.w[i] & 0x7fffffffu) : max_u16x2(most, e.w[i] & 0x7fff7fffu);
    return most;
}
template <typename T>
__device__ __forceinline__ uint32_t most2(uint32_t a, uint32_t b)
{
    return sizeof(T) == 4 ? max(a, b) : max_u16x2(a, b);
}
// The maximum as a number (infinite or NaN if any value is).
template <typename T>
__device__ __forceinline__ float most_value(uint32_t most)
{
    if constexpr (sizeof(T) == 4) {
        return __uint_as_float(most);
    } else {
        Run<T> e{};
        e.w[0] = max(most & 0xffffu, most >> 16);
        return pair_of(e, 0).x;
    }
}

__device__ __forceinline__ float step_of(float most)
{
    const float s = __fdiv_rn(most, 448.f);
    return s == 0.f ? 1.f : s;
}

// The codes of a run; rs: 1 / s correctly rounded.
template <typename T>
__device__ __forceinline__ void store_codes(uint8_t *row, int c, int cols, const Run<T> &e, float s, float rs)
{
    // div_rn_recip is exact for steps in [2^-60, 2^60] wherever the code is not zero
    const bool fast = s >= 0x1p-60f && s <= 0x1p60f;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 a = pair_of(e, 2 * i), b = pair_of(e, 2 * i + 1);
        if (fast) {
            a = make_float2(div_rn_recip(a.x, s, rs), div_rn_recip(a.y, s, rs));
            b = make_float2(div_rn_recip(b.x, s, rs), div_rn_recip(b.y, s, rs));
        } else {
            a = make_float2(__fdiv_rn(a.x, s), __fdiv_rn(a.y, s));
            b = make_float2(__fdiv_rn(b.x, s), __fdiv_rn(b.y, s));
        }
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    if (c + 16 <= cols) {
        *(uint4 *)(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (c + i < cols) row[c + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}

// One step per row and 128 columns.  A warp takes 1024 columns of one row (the
// grid's x: eight rows a CTA, y: strips of columns): 8 threads per block of 16
// values each, two blocks per thread in flight.  Bound by its bytes (4 + 1 or
// 2 + 1 per value) once each value takes few enough instructions: with eight
// values a thread and the steps computed by every lane it issued 19 per value
// and took 95 us for 16384 x 4096 in bf16, now 41 us (4.9 TB/s).  Six CTAs an
// SM for 16-bit values; for fp32 the registers that leaves (40) cost more than
// the occupancy gives: 37 us against 32 for 8000 x 4096.
constexpr int kStrip = 1024;
template <typename T>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 6 : 3) quantize_rows_kernel(const QuantArgs a)
{
    // (columns fit 32 bits: at most 2^30)
    const int cols = (int)a.cols, kblocks = (cols + 127) / 128, strips = (cols + kStrip - 1) / kStrip;
    const int lane = threadIdx.x & 31, sub = lane & 7;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= a.batch * a.rows) return;
    const int64_t e = a.batch > 1 ? row / a.rows : 0, r = row - e * a.rows;
    const T *src = (const T *)a.x + e * a.x_batch_stride + r * a.x_row_stride;
    uint8_t *dst = a.q + row * a.q_row_stride;
    float *steps = a.steps + row * kblocks;
    const int align = row_align(src);
    bool finite = true;
    for (int strip = blockIdx.y; strip < strips; strip += gridDim.y) {
        Run<T> v[2];
        uint32_t most[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = load_run(src, strip * kStrip + i * 512 + lane * 16, cols, align);
#pragma unroll
        for (int i = 0; i < 2; ++i) most[i] = most_of(v[i], 0u);
#pragma unroll
        for (int o = 4; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < 2; ++i) most[i] = most2<T>(most[i], __shfl_xor_sync(0xffffffffu, most[i], o));
        // the warp's eight steps: one per lane, then handed round
        const float m = most_value<T>(sub & 1 ? most[1] : most[0]), s_own = step_of(m), rs_own = __frcp_rn(s_own);
        finite &= isfinite(m);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float s = __shfl_sync(0xffffffffu, s_own, (lane & 24) | i);
            const float rs = __shfl_sync(0xffffffffu, rs_own, (lane & 24) | i);
            const int kb = strip * (kStrip / 128) + i * 4 + (lane >> 3);
            if (kb < kblocks) {
                store_codes(dst, kb * 128 + sub * 16, cols, v[i], s, rs);
                if (sub == 0) steps[kb] = s;
            }
        }
    }
    if (!finite) record_error(a.st, BAKRON_ERR_NONFINITE, (int)blockIdx.x);
}

// One step per 128 x 128 tile: one CTA per tile, its values in registers
// between the two passes.  14336 x 4096 in fp32: 53 us, 5.5 TB/s; with 256
// threads a CTA, and so half the loads in flight, 82 us.
constexpr int kTileThreads = 512, kTileRows = kTileThreads / 8, kTileLoads = 128 / kTileRows;
template <typename T>
__global__ void __launch_bounds__(kTileThreads, 2) quantize_tiles_kernel(const QuantArgs a)
{
    __shared__ uint32_t part[kTileThreads / 32];
    const unsigned kblocks = (unsigned)((a.cols + 127) / 128), rblocks = (unsigned)((a.rows + 127) / 128);
    const unsigned kb = blockIdx.x % kblocks, eb = blockIdx.x / kblocks, e = eb / rblocks, rb = eb - e * rblocks;
    const int sub = threadIdx.x & 7, r0 = threadIdx.x >> 3;
    const T *src = (const T *)a.x + e * a.x_batch_stride;
    const int align = min(row_align(src), row_align((const void *)(uintptr_t)(a.x_row_stride * (int64_t)sizeof(T))));
    const int c = (int)(kb * 128 + sub * 16);
    Run<T> v[kTileLoads];
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kTileLoads; ++i) {
        const int64_t r = (int64_t)rb * 128 + r0 + kTileRows * i;
        v[i] = load_run(src + r * a.x_row_stride, c, r < a.rows ? (int)a.cols : 0, align);
    }
#pragma unroll
    for (int i = 0; i < kTileLoads; ++i) most = most_of(v[i], most);
#pragma unroll
    for (int o = 16; o; o >>= 1) most = most2<T>(most, __shfl_xor_sync(0xffffffffu, most, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTileThreads / 32; ++i) most = most2<T>(most, part[i]);
    const float m = most_value<T>(most);
    if (!isfinite(m) && threadIdx.x == 0) record_error(a.st, BAKRON_ERR_NONFINITE, (int)blockIdx.x);
    const float s = step_of(m), rs = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < kTileLoads; ++i) {
        const int64_t r = (int64_t)rb * 128 + r0 + kTileRows * i;
        if (r < a.rows) store_codes(a.q + ((int64_t)e * a.rows + r) * a.q_row_stride, c, (int)a.cols, v[i], s, rs);
    }
    if (threadIdx.x == 0) a.steps[(int64_t)eb * kblocks + kb] = s;
}

template <typename T>
cudaError_t launch_typed(const QuantArgs &a, cudaStream_t stream)
{
    const int64_t kblocks = (a.cols + 127) / 128;
    if (a.block_rows == 1) {
        const dim3 grid((unsigned)((a.batch * a.rows + 7) / 8), (unsigned)min64((a.cols + kStrip - 1) / kStrip, 65535));
        quantize_rows_kernel<T><<<grid, 256, 0, stream>>>(a);
    } else {
        const int64_t blocks = a.batch * ((a.rows + 127) / 128) * kblocks;
        quantize_tiles_kernel<T><<<(unsigned)blocks, kTileThreads, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize(const QuantArgs &a, cudaStream_t stream)
{
    if (a.type == BAKRON_F32) return launch_typed<float>(a, stream);
    if (a.type == BAKRON_BF16) return launch_typed<__nv_bfloat16>(a, stream);
    return launch_typed<__half>(a, stream);
}

}  // namespace mm
}  // namespace bakron
