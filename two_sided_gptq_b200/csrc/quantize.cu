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

// Eight consecutive values of a row, as loaded.
template <typename T>
struct alignas(16) Eight {
    uint32_t w[8 * sizeof(T) / 4];
};

// From column c on, zeros from column `cols` on.
template <typename T>
__device__ __forceinline__ Eight<T> load8(const T *row, int c, int cols, bool vec)
{
    Eight<T> v;
    if (vec && c + 8 <= cols) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(v.w) / 16; ++i) ((uint4 *)v.w)[i] = __ldg((const uint4 *)(row + c) + i);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v.w[i] = c + i < cols ? __float_as_uint(row[c + i]) : 0u;
    } else {
        const uint16_t *h = (const uint16_t *)row;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = c + 2 * i < cols ? h[c + 2 * i] : 0u, hi = c + 2 * i + 1 < cols ? h[c + 2 * i + 1] : 0u;
            v.w[i] = lo | (hi << 16);
        }
    }
    return v;
}

__device__ __forceinline__ void to_floats(const Eight<float> &e, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(e.w[i]);
}
__device__ __forceinline__ void to_floats(const Eight<__nv_bfloat16> &e, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(e.w[i] << 16);
        v[2 * i + 1] = __uint_as_float(e.w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void to_floats(const Eight<__half> &e, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*(const __half2 *)&e.w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t m;
    asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
}

// The largest magnitude of the eight values and `most`, as the bits of the type
// with the sign cleared: ordered like the magnitudes, infinities and NaN above
// every finite value.  16-bit types keep two maxima in one word.
template <typename T>
__device__ __forceinline__ uint32_t most_of(const Eight<T> &e, uint32_t most)
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
        Eight<T> e{};
        e.w[0] = max(most & 0xffffu, most >> 16);
        float v[8];
        to_floats(e, v);
        return v[0];
    }
}

__device__ __forceinline__ float step_of(float most)
{
    const float s = __fdiv_rn(most, 448.f);
    return s == 0.f ? 1.f : s;
}

// rs: 1 / s correctly rounded.
template <typename T>
__device__ __forceinline__ void store8(uint8_t *row, int c, int cols, const Eight<T> &e, float s, float rs)
{
    float v[8];
    to_floats(e, v);
    // div_rn_recip is exact for steps in [2^-60, 2^60] wherever the code is not zero
    if (s >= 0x1p-60f && s <= 0x1p60f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = div_rn_recip(v[i], s, rs);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __fdiv_rn(v[i], s);
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi =
            __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    if (c + 8 <= cols) {
        *(uint2 *)(row + c) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) row[c + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}

// One step per row and 128 columns.  A warp takes 1024 columns of one row (the
// grid's x: eight rows a CTA, y: strips of columns): 16 threads per block of 8
// values each, four blocks in flight per thread.
constexpr int kStrip = 1024;
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantArgs a)
{
    // (columns fit 32 bits: at most 2^30)
    const int cols = (int)a.cols, kblocks = (cols + 127) / 128, strips = (cols + kStrip - 1) / kStrip;
    const int lane = threadIdx.x & 31, sub = lane & 15;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= a.batch * a.rows) return;
    const int64_t e = a.batch > 1 ? row / a.rows : 0, r = row - e * a.rows;
    const T *src = (const T *)a.x + e * a.x_batch_stride + r * a.x_row_stride;
    uint8_t *dst = a.q + row * a.q_row_stride;
    float *steps = a.steps + row * kblocks;
    const bool vec = ((uintptr_t)src & 15) == 0;
    bool finite = true;
    for (int strip = blockIdx.y; strip < strips; strip += gridDim.y) {
        Eight<T> v[4];
        uint32_t most[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = load8(src, strip * kStrip + i * 256 + lane * 8, cols, vec);
#pragma unroll
        for (int i = 0; i < 4; ++i) most[i] = most_of(v[i], 0u);
#pragma unroll
        for (int o = 8; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) most[i] = most2<T>(most[i], __shfl_xor_sync(0xffffffffu, most[i], o));
        // the warp's eight steps: one per lane, then handed round (computed by
        // every lane for itself, the divisions were a third of the instructions)
        const uint32_t own = sub & 2 ? (sub & 1 ? most[3] : most[2]) : (sub & 1 ? most[1] : most[0]);
        const float m = most_value<T>(own), s_own = step_of(m), rs_own = __frcp_rn(s_own);
        finite &= isfinite(m);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float s = __shfl_sync(0xffffffffu, s_own, (lane & 16) | i);
            const float rs = __shfl_sync(0xffffffffu, rs_own, (lane & 16) | i);
            const int kb = strip * (kStrip / 128) + i * 2 + (lane >> 4);
            if (kb < kblocks) {
                store8(dst, kb * 128 + sub * 8, cols, v[i], s, rs);
                if (sub == 0) steps[kb] = s;
            }
        }
    }
    if (!finite) record_error(a.st, BAKRON_ERR_NONFINITE, (int)blockIdx.x);
}

// One step per 128 x 128 tile: one CTA per tile, its values in registers
// between the two passes.
constexpr int kTileThreads = 512, kTileRows = kTileThreads / 16, kTileLoads = 128 / kTileRows;
template <typename T>
__global__ void __launch_bounds__(kTileThreads, 2) quantize_tiles_kernel(const QuantArgs a)
{
    __shared__ uint32_t part[kTileThreads / 32];
    const unsigned kblocks = (unsigned)((a.cols + 127) / 128), rblocks = (unsigned)((a.rows + 127) / 128);
    const unsigned kb = blockIdx.x % kblocks, eb = blockIdx.x / kblocks, e = eb / rblocks, rb = eb - e * rblocks;
    const int sub = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    const T *src = (const T *)a.x + e * a.x_batch_stride;
    const bool vec = (((uintptr_t)src | (uintptr_t)(a.x_row_stride * (int64_t)sizeof(T))) & 15) == 0;
    const int c = (int)(kb * 128 + sub * 8);
    Eight<T> v[kTileLoads];
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kTileLoads; ++i) {
        const int64_t r = (int64_t)rb * 128 + r0 + kTileRows * i;
        v[i] = load8(src + r * a.x_row_stride, c, r < a.rows ? (int)a.cols : 0, vec);
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
        if (r < a.rows) store8(a.q + ((int64_t)e * a.rows + r) * a.q_row_stride, c, (int)a.cols, v[i], s, rs);
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
