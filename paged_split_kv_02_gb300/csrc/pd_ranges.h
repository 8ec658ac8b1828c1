// Whole-number arithmetic of tiles, for the kernels and for checks on the host.
#pragma once

#include <climits>

#ifdef __CUDACC__
#define PD_BOTH __host__ __device__ __forceinline__
#else
#define PD_BOTH inline
#endif

namespace pd {

// May a work item name this tile: its rows [tile * rows, (tile + 1) * rows) are
// ints (the largest tile's end is, too, so that no sum with it wraps).
PD_BOTH bool tile_in_range(int tile, int rows) { return tile >= 0 && tile <= INT_MAX / rows - 1; }

}  // namespace pd
