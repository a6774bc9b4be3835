// mm_rows.cu -- products grouped by expert over packed rows, 16-bit operands:
// y[t, :] = x[t, :] w_e^T and dx[t, :] = dy[t, :] w_e (the weight read
// column-major there, through the MMA's transpose bit, so one copy of w serves
// both directions).
#include "mm_kernel.cuh"

namespace bakron {
namespace mm {

namespace {
template <int BN, bool AColumns>
struct Rows {
    static constexpr Ragged kRagged = kTokensB;
    static constexpr bool kPair = BN == 256, kEight = false, kAColumns = AColumns, kLower = false;
    static constexpr int kBN = BN, kPlanes = 1, kKRows = 0;
    static constexpr int kBoxRows = BN == 256 ? 64 : 32;
};
}  // namespace

cudaError_t configure_rows()
{
    cudaError_t e = configure<Rows<256, false>>();
    if (e == cudaSuccess) e = configure<Rows<64, false>>();
    if (e == cudaSuccess) e = configure<Rows<256, true>>();
    if (e == cudaSuccess) e = configure<Rows<64, true>>();
    return e;
}

cudaError_t launch_rows(Variant v, const Maps &maps, const Args &g, int64_t tiles, int sms,
                        cudaStream_t stream)
{
    switch (v) {
    case kRows256: return launch<Rows<256, false>>(maps, g, tiles, sms, stream);
    case kRows64: return launch<Rows<64, false>>(maps, g, tiles, sms, stream);
    case kRowsDx256: return launch<Rows<256, true>>(maps, g, tiles, sms, stream);
    default: return launch<Rows<64, true>>(maps, g, tiles, sms, stream);
    }
}

}  // namespace mm
}  // namespace bakron
