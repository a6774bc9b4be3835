// mm_outer.cu -- products whose contraction is the packed rows of a group: the
// experts' weight gradients dw_e = dy_e^T x_e, and one Gram factor per expert,
// A_e = X_e^T X_e / N_e + damping * mean(diag) * I (the K-FAC factor of an
// expert's inputs or output gradients, "Assumptions & free parameters": Gram
// matrix regularisation).
//
// FP32 samples are split once into three bf16 parts, x = h + m + l to 2^-27 of
// x; the products hh + (hm + mh) + mm + (hl + lh) on the bf16 tensor cores cost
// what three TF32 products would and keep 24 bits instead of 21.
//
// Tiles are 256 x 256 (256 x 128 from three parts, whose two accumulators fill
// tensor memory) by CTA pairs, or 128 x 128 by one CTA, whose contraction up to
// eight CTAs may share, where there are few of the former; only those that reach the lower triangle are
// formed, the rest is their mirror image.  A tile costs its group's length, so
// groups are taken longest first in rounds that run forth and back.
// Measured: dw of 16384 rows, 8 experts, 4096 x 1024 into fp32 121 us (1.14
// PFLOP/s; 104 us without its stores); Gram factors of 4 experts at d = 4096
// from 16384 bf16 rows 266 us (220 without the stores: 268 MB, both halves of
// every matrix); 8 experts at d = 1024 from 8192 fp32 rows 73 us: 12 to split
// the samples, 51 for the products (by either tile), 5 for the damping.  By pairs
// and as it is chosen: dw 512 x 512 from 4096 rows 28.4 and 12.9 us; Gram factors
// of 2 experts at d = 384 from 30000 rows 80 and 22 us.
#include "mm_kernel.cuh"

namespace bakron {
namespace mm {

namespace {
template <bool Pair>
struct Outer {
    static constexpr Ragged kRagged = kContract;
    static constexpr bool kPair = Pair, kJoin = !Pair, kEight = false, kAColumns = true, kLower = false;
    static constexpr int kBN = Pair ? 256 : 128, kPlanes = 1, kKRows = 64, kBoxRows = 64;
};
template <int Planes, bool Pair>
struct Gram {
    static constexpr Ragged kRagged = kContract;
    static constexpr bool kPair = Pair, kJoin = !Pair, kEight = false, kAColumns = true, kLower = true;
    static constexpr int kBN = Planes > 1 || !Pair ? 128 : 256, kPlanes = Planes, kKRows = Planes > 1 ? 32 : 64, kBoxRows = kKRows;
};

// Three bf16 parts of an fp32 matrix, each rounded to nearest from what the
// earlier ones leave (those differences are exact in fp32).  A warp takes 256
// columns of a row (grid x: eight rows a CTA, y: strips of columns), eight per
// thread.  Bound by its 4 + 6 bytes per element.
__global__ void __launch_bounds__(256) split_three_kernel(const float *__restrict__ x, int64_t rows, int64_t d,
                                                          int64_t ldx, __nv_bfloat16 *__restrict__ out, int64_t ld)
{
    pdl_wait();
    pdl_trigger();
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), plane = rows * ld;
    if (row >= rows) return;
    const float *src = x + row * ldx;
    const bool vec = ((uintptr_t)src & 15) == 0;
    for (int64_t c = (int64_t)blockIdx.y * 256 + (threadIdx.x & 31) * 8; c < d; c += (int64_t)gridDim.y * 256) {
        float v[8];
        if (vec && c + 8 <= d) {
            *(float4 *)v = __ldg((const float4 *)(src + c));
            *(float4 *)(v + 4) = __ldg((const float4 *)(src + c + 4));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = c + i < d ? src[c + i] : 0.f;
        }
        // (a plane's rows are padded to eight columns)
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            __align__(16) __nv_bfloat16 h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[i] = __float2bfloat16_rn(v[i]);
                v[i] -= __bfloat162float(h[i]);
            }
            *(uint4 *)(out + p * plane + row * ld + c) = *(const uint4 *)h;
        }
    }
}

// One CTA per group: the mean of the diagonal (FP64, a fixed order), then
// damping times it on the diagonal.  A diagonal entry is a sum of squares, so
// it is NaN or infinite whenever the group's samples hold such a value (or
// their squares overflow): recorded as BAKRON_ERR_NONFINITE.
__global__ void gram_damp_kernel(float *__restrict__ A, int64_t d, float damping, DeviceStatus *st)
{
    pdl_wait();
    pdl_trigger();
    __shared__ double part[32];
    __shared__ float add_sh;
    float *a = A + (int64_t)blockIdx.x * d * d;
    double sum = 0.0;
    bool finite = true;
    for (int64_t i = threadIdx.x; i < d; i += blockDim.x) {
        const float v = a[i * d + i];
        finite &= isfinite(v);
        sum += (double)v;
    }
    if (!finite) record_error(st, BAKRON_ERR_NONFINITE, (int)blockIdx.x);
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int w = 0; w < (int)(blockDim.x >> 5); ++w) t += part[w];
        add_sh = (float)((double)damping * (t / (double)d));
    }
    __syncthreads();
    const float add = add_sh;
    for (int64_t i = threadIdx.x; i < d; i += blockDim.x) a[i * d + i] = __fadd_rn(a[i * d + i], add);
}
}  // namespace

cudaError_t configure_outer()
{
    cudaError_t e = configure<Outer<true>>();
    if (e == cudaSuccess) e = configure<Outer<false>>();
    if (e == cudaSuccess) e = configure<Gram<1, true>>();
    if (e == cudaSuccess) e = configure<Gram<1, false>>();
    if (e == cudaSuccess) e = configure<Gram<3, true>>();
    return e == cudaSuccess ? configure<Gram<3, false>>() : e;
}

cudaError_t clusters_that_fit(int p, int &n)
{
    using S = Shape<Outer<false>>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = p;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(&n, mm_kernel<Outer<false>>, &cfg);
}

cudaError_t launch_outer(Variant v, const Maps &maps, const Args &g, int64_t tiles, int sms,
                        cudaStream_t stream)
{
    switch (v) {
    case kOuterPair: return launch<Outer<true>>(maps, g, tiles, sms, stream);
    case kOuterOne: return launch<Outer<false>>(maps, g, tiles, sms, stream);
    case kGramPair: return launch<Gram<1, true>>(maps, g, tiles, sms, stream);
    case kGramOne: return launch<Gram<1, false>>(maps, g, tiles, sms, stream);
    case kGramThreePair: return launch<Gram<3, true>>(maps, g, tiles, sms, stream);
    default: return launch<Gram<3, false>>(maps, g, tiles, sms, stream);
    }
}

cudaError_t launch_split_three(const float *x, int64_t rows, int64_t d, int64_t ldx, uint16_t *planes, int64_t ld,
                               cudaStream_t stream)
{
    const dim3 grid((unsigned)((rows + 7) / 8), (unsigned)min64((d + 255) / 256, 65535));
    return launch_pdl(split_three_kernel, grid, dim3(256), 0, stream, x, rows, d, ldx,
                      (__nv_bfloat16 *)planes, ld);
}

cudaError_t launch_gram_damp(float *A, int64_t d, int experts, float damping, DeviceStatus *st, cudaStream_t stream)
{
    return launch_pdl(gram_damp_kernel, dim3(experts), dim3(1024), 0, stream, A, d, damping, st);
}

}  // namespace mm
}  // namespace bakron
