// Host replay of the tile numbering of the products over packed rows, with the
// library's own rules (csrc/mm_groups.h): group after group, as the kernels'
// numbering warp does 32 at a time.
#include <stdint.h>

#include "mm_groups.h"

using namespace bakron::mm;

// Row tiles that the device numbers for these bounds; rows_of[e] says whether
// group e has its rows.  alone != 0: by each group's own bounds only.
extern "C" int64_t replay(const int32_t *offsets, int experts, int rows, int tile, int alone, uint8_t *rows_of)
{
    int64_t tiles = 0;
    int reach = 0;
    for (int e = 0; e < experts; ++e) {
        const int lo = offsets[e], hi = offsets[e + 1];
        rows_of[e] = alone ? is_range(lo, hi, rows) : has_rows(lo, hi, rows, reach);
        if (is_range(lo, hi, rows) && hi > reach) reach = hi;
        if (rows_of[e]) tiles += (hi - lo + (int64_t)tile - 1) / tile;
    }
    return tiles;
}

// Row tiles that the host launches for.
extern "C" int64_t launched(int64_t rows, int64_t experts, int64_t tile) { return row_tiles(rows, experts, tile); }
