// mm_eight.cu -- products of 8-bit (e4m3) operands with fp32 steps for blocks
// of 128 along the contraction, dense or grouped by expert.
//
// One ring stage is one 128-long block of the contraction, so every
// accumulator chunk belongs to one step of each operand: the epilogue adds
// (row step x weight step) times the chunk into its FP32 registers.  That chain
// -- MMA, commit, read, add, hand the buffer back -- takes about 2000 clocks
// whatever the tile, so its chunks in flight set the rate: two of 256 columns
// or four of 128.  Measured per
// chunk (8192 x 14336 x 4096): 1004 clocks at 256 x 256 (512 at the MMA peak,
// 770 without the additions, 684 without reading the accumulators at all: the
// operand loads, 48 bytes per clock and SM), 602 at 256 x 128, 630 at 128 x 128.
// 0.49 ms, 1.97 PFLOP/s at 1.6 GHz under the power cap.  The additions are plain
// FP32 fused multiply-adds: the packed form took 3.2 clocks a warp for two
// columns, against 2 for two plain ones.
// Short groups put the packed rows on the columns (128 x 64 tiles, the weight's
// 128 rows on the lanes); one token through 4096 x 4096 takes 7.9 us in a graph,
// of which 2.6 us are its 16.8 MB.
#include "mm_kernel.cuh"

namespace bakron {
namespace mm {

namespace {
// (The single CTA's tile comes with and without the join of a split contraction:
// with it the compiler's additions of a chunk take 25% longer, 85 against 68 us
// for 4100 rows of 16 experts, 4096 x 2048.)
template <bool Pair, int BN, bool Join = false>
struct EightA {
    static constexpr Ragged kRagged = kTokensA;
    static constexpr bool kPair = Pair, kJoin = Join, kEight = true, kAColumns = false, kLower = false;
    static constexpr int kBN = BN, kPlanes = 1, kKRows = 0, kBoxRows = 0;
};
struct EightB {
    static constexpr Ragged kRagged = kTokensB;
    static constexpr bool kPair = false, kJoin = true, kEight = true, kAColumns = false, kLower = false;
    static constexpr int kBN = 64, kPlanes = 1, kKRows = 0, kBoxRows = 32;
};
}  // namespace

cudaError_t configure_eight()
{
    cudaError_t e = configure<EightA<true, 256>>();
    if (e == cudaSuccess) e = configure<EightA<true, 128>>();
    if (e == cudaSuccess) e = configure<EightA<false, 128>>();
    if (e == cudaSuccess) e = configure<EightA<false, 128, true>>();
    return e == cudaSuccess ? configure<EightB>() : e;
}

cudaError_t launch_eight(Variant v, const Maps &maps, const Args &g, int64_t tiles, int sms,
                        cudaStream_t stream)
{
    switch (v) {
    case kEightPair256: return launch<EightA<true, 256>>(maps, g, tiles, sms, stream);
    case kEightPair128: return launch<EightA<true, 128>>(maps, g, tiles, sms, stream);
    case kEightOne128:
        return g.split > 1 ? launch<EightA<false, 128, true>>(maps, g, tiles, sms, stream)
                           : launch<EightA<false, 128>>(maps, g, tiles, sms, stream);
    default: return launch<EightB>(maps, g, tiles, sms, stream);
    }
}

}  // namespace mm
}  // namespace bakron
