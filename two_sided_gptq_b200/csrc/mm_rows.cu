// mm_rows.cu -- products grouped by expert over packed rows, 16-bit operands:
// y[t, :] = x[t, :] w_e^T and dx[t, :] = dy[t, :] w_e (the weight read
// column-major there, through the MMA's transpose bit, so one copy of w serves
// both directions).
//
// Long groups: 256 x 256 tiles by CTA pairs, six 32 KB stages a CTA.  16384 rows
// of 8 experts, 4096 x 4096 (5.5e11 FLOP): 566 clocks a stage of 512 at the MMA
// peak, 0.37 ms (1.48 PFLOP/s) until the 1000 W power cap takes the clock from
// 1.6 to 1.27 GHz (0.45 ms, 1.2 PFLOP/s; the cuBLAS product of the same session
// sustained 1.3).  With one CTA a tile (128 x 256) it took 0.62 ms.
// Short groups (48 rows on average or fewer): 128 x 64 tiles, eight 24 KB
// stages, bound by reading the weights: 96 rows over 64 experts of 1024 x 2048
// (172 MB) take 35 us, 4.9 TB/s, in 2.5 rounds of tiles over the SMs.  With
// four stages, and so half the weights in flight, it took 38 us.
#include "mm_kernel.cuh"

namespace bakron {
namespace mm {

namespace {
template <int BN, bool AColumns>
struct Rows {
    static constexpr Ragged kRagged = kTokensB;
    static constexpr bool kPair = BN == 256, kJoin = !kPair, kEight = false, kAColumns = AColumns, kLower = false;
    static constexpr int kBN = BN, kPlanes = 1, kKRows = 0;
    static constexpr int kBoxRows = BN == 256 ? 64 : 32;
};
struct RowsAbort : Rows<256, false> {};
}  // namespace

template <>
constexpr bool kGivesUp<RowsAbort> = true;

cudaError_t configure_rows()
{
    cudaError_t e = configure<Rows<256, false>>();
    if (e == cudaSuccess) e = configure<Rows<64, false>>();
    if (e == cudaSuccess) e = configure<Rows<256, true>>();
    if (e == cudaSuccess) e = configure<Rows<64, true>>();
    if (e == cudaSuccess) e = configure<RowsAbort>();
    return e;
}

cudaError_t launch_rows(Variant v, const Maps &maps, const Args &g, int64_t tiles, int sms,
                        cudaStream_t stream)
{
    switch (v) {
    case kRows256: return launch<Rows<256, false>>(maps, g, tiles, sms, stream);
    case kRows64: return launch<Rows<64, false>>(maps, g, tiles, sms, stream);
    case kRowsDx256: return launch<Rows<256, true>>(maps, g, tiles, sms, stream);
    case kRowsAbort: return launch<RowsAbort>(maps, g, tiles, sms, stream);
    default: return launch<Rows<64, true>>(maps, g, tiles, sms, stream);
    }
}

}  // namespace mm
}  // namespace bakron
