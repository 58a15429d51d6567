// Which rows a block of a grouped product works on.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4 {

// Rows lo .. hi - 1 of y, hi the end of expert e's rows (not of the tile);
// e == experts: rows of no expert; e < 0: no such tile.
struct GroupTile {
  int32_t e, lo, hi;
};

// Inclusive scan over the wave's lanes (identity 0).
template <typename F>
__device__ __forceinline__ uint32_t wave_scan(uint32_t v, F&& op) {
  // row_shr 1, 2, 4, 8, then the last lane of each row of 16 (row_bcast 15)
  // and of each half (row_bcast 31) into the rows after it
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false));
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false));
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false));
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false));
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));
  return v;
}

// Tile t (the same in every lane) when each expert's rows, and at last the rows
// of no expert, are cut into tiles of ROWS.  Every lane of the wave calls it.
// 64 experts at a time, one a lane: the ends as a running maximum within
// [0, rows], so that no offsets lead out of the buffers, then the tiles' sums.
// A tile starts at row lo; the last tile of an expert may hold fewer rows.
template <int ROWS>
__device__ __forceinline__ GroupTile find_group_tile(const int32_t* offsets, int32_t experts,
                                                     int32_t rows, uint32_t t) {
  const int lane = threadIdx.x & 63;
  uint32_t before = 0, at = 0;  // tiles and rows of the experts seen
  for (int32_t c = 0; c <= experts; c += 64) {
    const int32_t e = c + lane;
    int32_t o = rows;
    if (e < experts) o = offsets[e + 1];
    o = o < 0 ? 0 : o > rows ? rows : o;
    uint32_t end = (uint32_t)o > at ? (uint32_t)o : at;
    end = wave_scan(end, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
    uint32_t lo = (uint32_t)__shfl_up((int)end, 1);
    if (lane == 0) lo = at;
    const uint32_t tiles = (end - lo + ROWS - 1) / ROWS;
    const uint32_t upto = before + wave_scan(tiles, [](uint32_t a, uint32_t b) { return a + b; });
    const uint64_t hit = __ballot(t < upto);
    if (hit) {
      const int f = __builtin_ctzll(hit);
      const uint32_t first = (uint32_t)__builtin_amdgcn_readlane((int)(upto - tiles), f);
      const int32_t l = __builtin_amdgcn_readlane((int)lo, f);
      return GroupTile{c + f, l + (int32_t)(t - first) * ROWS, __builtin_amdgcn_readlane((int)end, f)};
    }
    before = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
    at = (uint32_t)__builtin_amdgcn_readlane((int)end, 63);
  }
  return GroupTile{-1, 0, 0};
}

}  // namespace w4
