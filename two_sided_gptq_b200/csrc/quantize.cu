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

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

// Eight consecutive values from column c of a row, zeros from column `cols` on.
template <typename T>
__device__ __forceinline__ void load8(const T *row, int64_t c, int64_t cols, bool vec, float (&v)[8])
{
    if (vec && c + 8 <= cols) {
        __align__(16) T t[8];
        constexpr int kLoads = 8 * sizeof(T) / 16;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) ((uint4 *)t)[i] = __ldg((const uint4 *)(row + c) + i);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_float(t[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? to_float(row[c + i]) : 0.f;
    }
}

__device__ __forceinline__ float step_of(float most)
{
    const float s = __fdiv_rn(most, 448.f);
    return s == 0.f ? 1.f : s;
}

__device__ __forceinline__ void store8(uint8_t *row, int64_t c, int64_t cols, const float (&v)[8], float s)
{
    // div_rn_recip is exact for steps in [2^-60, 2^60] wherever the code is not zero
    const bool fast = s >= 0x1p-60f && s <= 0x1p60f;
    const float rs = __frcp_rn(s);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float q[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) q[u] = fast ? div_rn_recip(v[4 * i + u], s, rs) : __fdiv_rn(v[4 * i + u], s);
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[2], q[3]), __NV_SATFINITE, __NV_E4M3);
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

// One step per row and 128 columns: 16 threads per block of 8 values each.
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantArgs a)
{
    const int64_t kblocks = (a.cols + 127) / 128, total = a.batch * a.rows * kblocks;
    const int sub = threadIdx.x & 15;
    const bool vec = (((uintptr_t)a.x | (a.x_row_stride * sizeof(T)) | (a.x_batch_stride * sizeof(T))) & 15) == 0;
    bool finite = true;
    for (int64_t b = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 4; b - (threadIdx.x >> 4 & 1) < total;
         b += (int64_t)gridDim.x * 16) {
        const bool live = b < total;
        const int64_t row = live ? b / kblocks : 0, kb = live ? b - row * kblocks : 0;
        const int64_t e = row / a.rows, r = row - e * a.rows, c = kb * 128 + sub * 8;
        const T *src = (const T *)a.x + e * a.x_batch_stride + r * a.x_row_stride;
        float v[8];
        load8(src, c, live ? a.cols : 0, vec, v);
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            most = fmaxf(most, fabsf(v[i]));
            finite &= isfinite(v[i]);
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        const float s = step_of(most);
        if (live) {
            store8(a.q + row * a.q_row_stride, c, a.cols, v, s);
            if (sub == 0) a.steps[row * kblocks + kb] = s;
        }
    }
    if (!finite) record_error(a.st, BAKRON_ERR_NONFINITE, (int)blockIdx.x);
}

// One step per 128 x 128 tile: one CTA per tile, its values in registers
// between the two passes.
template <typename T>
__global__ void __launch_bounds__(256) quantize_tiles_kernel(const QuantArgs a)
{
    __shared__ float part[8];
    const int64_t kblocks = (a.cols + 127) / 128, rblocks = (a.rows + 127) / 128;
    const int64_t kb = blockIdx.x % kblocks, eb = blockIdx.x / kblocks, e = eb / rblocks, rb = eb - e * rblocks;
    const int sub = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    const bool vec = (((uintptr_t)a.x | (a.x_row_stride * sizeof(T)) | (a.x_batch_stride * sizeof(T))) & 15) == 0;
    const int64_t c = kb * 128 + sub * 8;
    float v[8][8], most = 0.f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = rb * 128 + r0 + 16 * i;
        load8((const T *)a.x + e * a.x_batch_stride + r * a.x_row_stride, c, r < a.rows ? a.cols : 0, vec, v[i]);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            most = fmaxf(most, fabsf(v[i][u]));
            finite &= isfinite(v[i][u]);
        }
    }
    if (!finite) record_error(a.st, BAKRON_ERR_NONFINITE, (int)blockIdx.x);
#pragma unroll
    for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) most = fmaxf(most, part[i]);
    const float s = step_of(most);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = rb * 128 + r0 + 16 * i;
        if (r < a.rows) store8(a.q + (e * a.rows + r) * a.q_row_stride, c, a.cols, v[i], s);
    }
    if (threadIdx.x == 0) a.steps[eb * kblocks + kb] = s;
}

template <typename T>
cudaError_t launch_typed(const QuantArgs &a, cudaStream_t stream)
{
    const int64_t kblocks = (a.cols + 127) / 128;
    if (a.block_rows == 1) {
        const int64_t blocks = min64((a.batch * a.rows * kblocks + 15) / 16, 148 * 8);
        quantize_rows_kernel<T><<<(unsigned)blocks, 256, 0, stream>>>(a);
    } else {
        const int64_t blocks = a.batch * ((a.rows + 127) / 128) * kblocks;
        quantize_tiles_kernel<T><<<(unsigned)blocks, 256, 0, stream>>>(a);
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
