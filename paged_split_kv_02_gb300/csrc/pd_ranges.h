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

// The keys [lo, hi) of a row's window: the row of token tok (below ml) of the ml
// new ones of a request of L keys, ml of them or fewer; window >= 1.  Nothing
// here wraps: a request may have fewer keys than new tokens, and a window be as
// long as an int.
struct RowKeys {
  int lo, hi;
};
PD_BOTH RowKeys row_keys(int L, int ml, int tok, int window) {
  const int n = L - ml + tok + 1, hi = n > 0 ? n : 0;
  return {hi > window ? hi - window : 0, hi};
}

}  // namespace pd
