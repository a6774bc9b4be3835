// mm.cuh -- launch interface of the products over packed rows (mm_kernel.cuh)
// and of the 8-bit block quantiser.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace bakron {
namespace mm {

enum Ragged { kTokensB, kTokensA, kContract };

constexpr int kMaxExperts = 1024;

struct Maps {
    CUtensorMap a, b;
    CUtensorMap b2;  // packed rows on D's columns: boxes of twice as many rows
};

struct Args {
    const int32_t *offsets;  // device, experts + 1 row bounds; NULL: one group of all rows
    int experts, rows;       // groups, packed rows
    int a_total, b_total;    // extents of D's rows / columns where they are not the packed rows
    int k_total;             // contraction where it is not the packed rows
    void *out;
    int64_t ldo, out_expert_stride;  // elements
    int out_type;                    // bakron_type_t
    int turn;                        // 16-bit result whose rows all start on 16-byte boundaries
    uint32_t idesc;                  // MMA instruction descriptor without M and N
    const float *x_steps, *w_steps;  // 8-bit operands' steps
    int w_step_rows;                 // rows per weight step: 128, or 1 (one step per row)
    int chunk;                       // stages per accumulator chunk (16-bit operands)
    int split;                       // CTAs that share a tile's contraction (kernels that can split)
    DeviceStatus *st;
    uint64_t timeout_ns;
    int gives_up;                    // self-test only
};

// A product of the library: which kernel variant runs it.
enum Variant {
    kRows256, kRows64,          // y = x w^T: packed rows on D's columns, tiles of 256 / 64
    kRowsDx256, kRowsDx64,      // dx = dy w
    kRowsAbort,                 // kRows256 with a wait that counts as run out (self-test)
    kOuterPair, kOuterOne,      // dw = dy^T x, by tiles of a CTA pair / of one CTA
    kGramPair, kGramOne,        // X^T X from 16-bit samples
    kGramThreePair, kGramThreeOne,  // X^T X from three bf16 parts of fp32 samples
    kEightPair256, kEightPair128, kEightOne128,  // 8-bit operands, packed rows on D's rows: 256 of them
                                                 // (a CTA pair) or 128, by 256 or 128 columns
    kEightB64                                    // packed rows on D's columns
};

cudaError_t configure_rows();
cudaError_t configure_eight();
cudaError_t configure_outer();
// How many clusters of p CTAs run at once (kernels whose contraction is split hold
// an SM per CTA, all alike).
cudaError_t clusters_that_fit(int p, int &n);
cudaError_t launch_rows(Variant v, const Maps &maps, const Args &g, int64_t tiles, int sms,
                        cudaStream_t stream);
cudaError_t launch_eight(Variant v, const Maps &maps, const Args &g, int64_t tiles, int sms,
                        cudaStream_t stream);
cudaError_t launch_outer(Variant v, const Maps &maps, const Args &g, int64_t tiles, int sms,
                        cudaStream_t stream);

// x ~= h + m + l in bf16, three planes of rows x ld; fp32 input with row stride ldx.
cudaError_t launch_split_three(const float *x, int64_t rows, int64_t d, int64_t ldx, uint16_t *planes, int64_t ld,
                               cudaStream_t stream);
// Damping of per-group Gram matrices: the diagonal gets damping times its mean.
cudaError_t launch_gram_damp(float *A, int64_t d, int experts, float damping, DeviceStatus *st, cudaStream_t stream);

// 8-bit block quantiser (quantize.cu).
struct QuantArgs {
    const void *x;
    int type;  // bakron_type_t
    int64_t batch, rows, cols, x_batch_stride, x_row_stride;
    int block_rows;  // 1 or 128
    uint8_t *q;
    int64_t q_row_stride;
    float *steps;
    DeviceStatus *st;
};
cudaError_t launch_quantize(const QuantArgs &a, cudaStream_t stream);

}  // namespace mm

// Row-major matrices as TMA tensor maps with 128-byte swizzle: dims[0] is the
// contiguous one, strides in bytes for dims[1..rank-1].
bool encode_tensor_map(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base, const uint64_t *dims,
                       const uint64_t *strides, const uint32_t *box);

}  // namespace bakron
