// mm_groups.h -- which packed rows a group has, and how many tiles of them a
// call has at most.  Plain functions of the row bounds, shared by the kernels
// (mm_kernel.cuh), the host's choice of a launch (mm_api.cu) and the host replay
// of the two (tests/cuda/group_replay.cpp).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define BAKRON_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define BAKRON_HOST_DEVICE inline
#endif

namespace bakron {
namespace mm {

// Bounds that are a range of the packed rows (an empty one included).
BAKRON_HOST_DEVICE bool is_range(int lo, int hi, int rows) { return lo >= 0 && lo <= hi && hi <= rows; }

// Whether a group gets the rows between its bounds.  `reach` is the largest end
// of the ranges before it (0 without one): bounds that go back to rows behind it
// would give the same rows to two groups.  So the groups that count share no row,
// which row_tiles() relies on.
BAKRON_HOST_DEVICE bool has_rows(int lo, int hi, int rows, int reach) { return is_range(lo, hi, rows) && lo >= reach; }

// Tiles of `tile` packed rows that the groups of a call have at most: every
// group adds at most one partial tile, and a group without rows adds none.
BAKRON_HOST_DEVICE int64_t row_tiles(int64_t rows, int64_t experts, int64_t tile)
{
    return rows / tile + (experts < rows ? experts : rows);
}

}  // namespace mm
}  // namespace bakron
