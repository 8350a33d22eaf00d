// Row tiles of sorted rows: which bin a tile lies in (device code shared by the
// kernels that walk rows sorted by wq_sort_rows).
#pragma once

#include "wq_internal.h"

namespace wq {

struct RowTile {
  int bin;    // its bin; bins for the tail behind the last one
  int row0;   // first sorted row
  int rows;   // rows in the tile, at least 1
};

// Inclusive sum over the wave's lanes, in the vector units' own lane moves (row
// shifts by 1, 2, 4, 8, then the last lanes of rows 0, 2 and of the lower half
// to the rows after them): no LDS round trip.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);
  return x;
}

// Tile m of the sorted rows (bins 0 .. bins - 1, and with TAIL the rows behind
// them up to `slots` as one more).  Called by whole waves: every lane takes
// one bin of 64 at a time, a wave scan numbers the tiles.  Offsets are clamped
// to 0 .. slots, so no plan leads outside the rows.  Returns false if there are
// not that many tiles; *count gets their number.
template <bool TAIL>
__device__ __forceinline__ bool find_row_tile(const int* __restrict__ offsets, int bins, int slots, int shift, int m,
                                              RowTile& tile, int& count) {
  const int lane = threadIdx.x & 63;
  const int nb = bins + (TAIL ? 1 : 0);
  int run = 0;
  bool found = false;
  for (int c = 0; c < nb; c += 64) {
    const int b = c + lane;
    int lo = 0, hi = 0;
    if (b < nb) {
      lo = min(max(offsets[b], 0), slots);
      hi = TAIL && b == bins ? slots : min(max(offsets[b + 1], lo), slots);
    }
    const int tiles = (hi - lo + (1 << shift) - 1) >> shift;
    const int incl = wave_scan(tiles);
    const int sum = __builtin_amdgcn_readlane(incl, 63);
    if (!found && m < run + sum) {
      const int l = __ffsll((unsigned long long)__ballot(incl > m - run)) - 1;
      const int first = __builtin_amdgcn_readlane(lo, l), last = __builtin_amdgcn_readlane(hi, l);
      const int before = run + __builtin_amdgcn_readlane(incl - tiles, l);
      tile.bin = c + l;
      tile.row0 = first + ((m - before) << shift);
      tile.rows = min(1 << shift, last - tile.row0);
      found = true;
    }
    run += sum;
  }
  count = run;
  return found;
}

// The number of row tiles alone (whole waves, as above).
__device__ __forceinline__ int count_row_tiles(const int* __restrict__ offsets, int bins, int slots, int shift) {
  const int lane = threadIdx.x & 63;
  int tiles = 0;
  for (int b = lane; b < bins; b += 64) {
    const int lo = min(max(offsets[b], 0), slots), hi = min(max(offsets[b + 1], lo), slots);
    tiles += (hi - lo + (1 << shift) - 1) >> shift;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) tiles += __shfl_xor(tiles, d);
  return __builtin_amdgcn_readfirstlane(tiles);
}

}  // namespace wq
