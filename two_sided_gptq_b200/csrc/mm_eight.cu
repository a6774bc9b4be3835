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
template <bool Pair, int BN>
struct EightA {
    static constexpr Ragged kRagged = kTokensA;
    static constexpr bool kPair = Pair, kEight = true, kAColumns = false, kLower = false;
    static constexpr int kBN = BN, kPlanes = 1, kKRows = 0, kBoxRows = 0;
};
struct EightB {
    static constexpr Ragged kRagged = kTokensB;
    static constexpr bool kPair = false, kEight = true, kAColumns = false, kLower = false;
    static constexpr int kBN = 64, kPlanes = 1, kKRows = 0, kBoxRows = 32;
};
}  // namespace

cudaError_t configure_eight()
{
    cudaError_t e = configure<EightA<true, 256>>();
    if (e == cudaSuccess) e = configure<EightA<true, 128>>();
    if (e == cudaSuccess) e = configure<EightA<false, 128>>();
    return e == cudaSuccess ? configure<EightB>() : e;
}

cudaError_t launch_eight(Variant v, const Maps &maps, const Args &g, int64_t tiles, int sms,
                        cudaStream_t stream)
{
    switch (v) {
    case kEightPair256: return launch<EightA<true, 256>>(maps, g, tiles, sms, stream);
    case kEightPair128: return launch<EightA<true, 128>>(maps, g, tiles, sms, stream);
    case kEightOne128: return launch<EightA<false, 128>>(maps, g, tiles, sms, stream);
    default: return launch<EightB>(maps, g, tiles, sms, stream);
    }
}

}  // namespace mm
}  // namespace bakron
