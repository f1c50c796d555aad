// raster.hpp -- which tile of a GEMM-shaped launch a workgroup takes (internal).
#pragma once

#include <hip/hip_runtime.h>

namespace grpo {

// Logical tile id p -> (M-tile, N-tile), in groups of GM M-tiles (M
// fastest), so the ~32 workgroups resident on one XCD share GM A-panels and
// ~32/GM B-panels in that XCD's L2.
template <int GM>
__device__ __forceinline__ void group_coords(int p, int tm, int tn, int& mt, int& nt) {
  const int per_group = GM * tn;
  const int g = p / per_group;
  const int first = g * GM;
  const int gm = (tm - first) < GM ? (tm - first) : GM;
  const int rem = p - g * per_group;
  mt = first + rem % gm;
  nt = rem / gm;
}

// Hardware dispatches workgroup b to XCD b % 8.  Deal the logical tile ids
// [0, tiles) to the XCDs in whole blocks of 32, one wave of an XCD's 32 CUs:
// XCD x takes a contiguous range of blocks, so the tiles resident on it at
// one time are always one aligned block of the raster.  (A range starting
// part-way into a block would straddle two groups of the raster for some of
// its waves.)  The grid is xcd_grid(tiles) workgroups; false for those past
// this XCD's range.
__device__ __forceinline__ bool xcd_tile(int bid, int tiles, int& p) {
  const int xcd = bid & 7, slot = bid >> 3;
  const int nb = (tiles + 31) >> 5;
  const int q = nb >> 3, r = nb & 7;
  const int nmine = (q + (xcd < r ? 1 : 0)) << 5;
  p = ((xcd * q + (xcd < r ? xcd : r)) << 5) + slot;
  return slot < nmine && p < tiles;
}

}  // namespace grpo
