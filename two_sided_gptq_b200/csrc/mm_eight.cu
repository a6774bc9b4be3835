// mm_eight.cu -- products of 8-bit (e4m3) operands with fp32 steps for blocks
// of 128 along the contraction, dense or grouped by expert.
//
// One ring stage is one 128-long block of the contraction, so every
// accumulator chunk belongs to one step of each operand: the epilogue adds
// (row step x weight step) times the chunk into its FP32 registers.
#include "mm_kernel.cuh"

namespace bakron {
namespace mm {

namespace {
struct EightA {
    static constexpr Ragged kRagged = kTokensA;
    static constexpr bool kPair = true, kEight = true, kAColumns = false, kLower = false;
    static constexpr int kBN = 256, kPlanes = 1, kKRows = 0, kBoxRows = 128;
};
struct EightB {
    static constexpr Ragged kRagged = kTokensB;
    static constexpr bool kPair = false, kEight = true, kAColumns = false, kLower = false;
    static constexpr int kBN = 64, kPlanes = 1, kKRows = 0, kBoxRows = 32;
};
}  // namespace

cudaError_t configure_eight()
{
    cudaError_t e = configure<EightA>();
    return e == cudaSuccess ? configure<EightB>() : e;
}

cudaError_t launch_eight(Variant v, const Maps &maps, const Args &g, int64_t tiles, int sms,
                        cudaStream_t stream)
{
    return v == kEightA256 ? launch<EightA>(maps, g, tiles, sms, stream) : launch<EightB>(maps, g, tiles, sms, stream);
}

}  // namespace mm
}  // namespace bakron
