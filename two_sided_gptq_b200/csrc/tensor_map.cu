// tensor_map.cu -- TMA tensor maps (cuTensorMapEncodeTiled, looked up in the
// driver at run time so that the library links without libcuda).
#include <cuda.h>
#include <cuda_runtime.h>

#include "mm.cuh"

namespace bakron {

namespace {
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn find_encode()
{
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
        return (EncodeTiledFn)p;
    return nullptr;
}
}  // namespace

bool encode_tensor_map(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base, const uint64_t *dims,
                       const uint64_t *strides, const uint32_t *box)
{
    static const EncodeTiledFn enc = find_encode();
    if (!enc) return false;
    cuuint64_t d[3] = {1, 1, 1}, s[2] = {0, 0};
    cuuint32_t b[3] = {1, 1, 1};
    const cuuint32_t elem[3] = {1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        if (i + 1 < rank) s[i] = strides[i];
    }
    return enc(map, type, (cuuint32_t)rank, (void *)base, d, s, b, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace bakron
