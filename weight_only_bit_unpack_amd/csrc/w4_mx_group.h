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

// The tiles when each expert's rows, and at last the rows of no expert, are cut
// into tiles of ROWS.  A tile starts at row lo; the last one of an expert may
// hold fewer rows.  The ends are read as a running maximum within [0, rows], so
// that no offsets lead out of the buffers.  Every lane of the wave calls these,
// read() first.
template <int ROWS>
struct GroupScan {
  const int32_t* offsets;
  int32_t experts, rows;
  uint32_t lo0 = 0, end0 = 0, upto0 = 0;  // the first 64 experts, once read

  __device__ __forceinline__ GroupScan(const int32_t* o, int32_t e, int32_t r) : offsets(o), experts(e), rows(r) {}
  __device__ __forceinline__ void read() { chunk(0, 0, 0, lo0, end0, upto0); }

  // 64 experts from c on, one a lane: before, at -- tiles and rows of the
  // experts before c.  lo, end: the expert's rows; upto: tiles up to and with it.
  __device__ __forceinline__ void chunk(int32_t c, uint32_t before, uint32_t at, uint32_t& lo, uint32_t& end,
                                        uint32_t& upto) const {
    const int lane = threadIdx.x & 63;
    const int32_t e = c + lane;
    int32_t o = rows;
    if (e < experts) o = offsets[e + 1];
    o = o < 0 ? 0 : o > rows ? rows : o;
    end = (uint32_t)o > at ? (uint32_t)o : at;
    end = wave_scan(end, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
    lo = (uint32_t)__shfl_up((int)end, 1);
    if (lane == 0) lo = at;
    upto = before + wave_scan((end - lo + ROWS - 1) / ROWS, [](uint32_t a, uint32_t b) { return a + b; });
  }

  // tile t, the same in every lane
  __device__ __forceinline__ GroupTile find(uint32_t t) const {
    uint32_t before = 0, at = 0;
    GroupTile g{-1, 0, 0};
    for (int32_t c = 0; c <= experts; c += 64) {
      uint32_t lo = lo0, end = end0, upto = upto0;
      if (c > 0) chunk(c, before, at, lo, end, upto);
      const uint64_t hit = __ballot(t < upto);
      if (hit) {
        const int f = __builtin_ctzll(hit);
        const uint32_t first =
            (uint32_t)__builtin_amdgcn_readlane((int)(upto - (end - lo + ROWS - 1) / ROWS), f);
        g = GroupTile{c + f, __builtin_amdgcn_readlane((int)lo, f) + (int32_t)(t - first) * ROWS,
                      __builtin_amdgcn_readlane((int)end, f)};
        break;
      }
      before = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
      at = (uint32_t)__builtin_amdgcn_readlane((int)end, 63);
    }
    // (the same in every lane: the addresses made from it stay scalar)
    return GroupTile{__builtin_amdgcn_readfirstlane(g.e), __builtin_amdgcn_readfirstlane(g.lo),
                     __builtin_amdgcn_readfirstlane(g.hi)};
  }

  // the number of tiles
  __device__ __forceinline__ uint32_t count() const {
    uint32_t before = 0, at = 0;
    for (int32_t c = 0; c <= experts; c += 64) {
      uint32_t lo = lo0, end = end0, upto = upto0;
      if (c > 0) chunk(c, before, at, lo, end, upto);
      before = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
      at = (uint32_t)__builtin_amdgcn_readlane((int)end, 63);
    }
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)before);
  }
};

}  // namespace w4
