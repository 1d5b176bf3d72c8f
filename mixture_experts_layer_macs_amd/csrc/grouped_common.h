// Ragged groups of rows: which expert and which of its rows a tile of a grouped
// product covers, found on the device from the expert offsets.
#pragma once

#include "common.h"

namespace moe {
namespace grp {

struct Groups {
  const int32_t* offsets;  // [N+1]
  int N, R;                // R: rows that the arrays hold
};

struct Span {
  int lo, hi;  // rows of an expert
};

// Held inside [0, R] whatever the offsets are, so that no row outside the
// arrays is touched.
__device__ __forceinline__ Span span_of(const Groups& g, int e) {
  const int lo = max(0, min(g.offsets[e], g.R));
  return {lo, max(lo, min(g.offsets[e + 1], g.R))};
}

struct RowTile {
  int e, lo, hi;  // the expert and its rows
  int tile;       // tile among the expert's; e == -1: past the last tile
  int before;     // tiles of the experts before it
};

// Tile `at` of the list of all experts' row tiles of `height` rows.  A wave's
// work, all lanes active, the same result in every lane: 64 experts at a time
// are scanned with their tile counts in the lanes.
__device__ __forceinline__ RowTile row_tile(const Groups& g, int height, int at) {
  const int lane = lane_id();
  int before = 0;
  for (int e0 = 0; e0 < g.N; e0 += MOE_WAVE) {
    const int e = e0 + lane;
    const Span s = span_of(g, min(e, g.N - 1));
    const int tiles = e < g.N ? (s.hi - s.lo + height - 1) / height : 0;
    const int incl = before + wave_incl_scan(tiles);
    const uint64_t past = __ballot(incl > at);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int first = read_lane(incl - tiles, l);
      return {e0 + l, read_lane(s.lo, l), read_lane(s.hi, l), at - first, first};
    }
    before = read_lane(incl, MOE_WAVE - 1);
  }
  return {-1, 0, 0, 0, before};
}

// All experts' row tiles of `height` rows; a wave's work as above.
__device__ __forceinline__ int row_tiles(const Groups& g, int height) {
  int n = 0;
  for (int e = lane_id(); e < g.N; e += MOE_WAVE) {
    const Span s = span_of(g, e);
    n += (s.hi - s.lo + height - 1) / height;
  }
  return wave_sum(n);
}

// Workgroups go round-robin over the 8 XCDs: place `block` of a list of `total`
// tiles of which each XCD gets one contiguous range; -1: none.
__device__ __forceinline__ int place_of(int block, int total) {
  const int q = (total + 7) / 8, at = block % 8 * q + block / 8;
  return block / 8 < q && at < total ? at : -1;
}

// Tile `in` of rows x cols tiles, in bands of at most 6 rows, so that tiles that
// run side by side share the operands' slices in the XCD's L2.
__device__ __forceinline__ void banded(int in, int rows, int cols, int& mt, int& nt) {
  const int bands = (rows + 5) / 6, height = (rows + bands - 1) / bands;
  const int band = in / (height * cols), at = in - band * height * cols;
  const int h = min(height, rows - band * height);
  mt = band * height + at % h;
  nt = at / h;
}

// Tile of a product of data rows: expert by expert.
__device__ __forceinline__ bool data_tile(const Groups& g, int height, int cols, int block, int& e,
                                          int& lo, int& hi, int& mt, int& nt) {
  const int at = place_of(block, row_tiles(g, height) * cols);
  if (at < 0) return false;
  const RowTile t = row_tile(g, height, at / cols);
  e = t.e;
  lo = t.lo;
  hi = t.hi;
  banded(at - t.before * cols, (hi - lo + height - 1) / height, cols, mt, nt);
  return true;
}

// Tile of a weight gradient, and part of its reduction.
__device__ __forceinline__ bool weight_tile(int N, int rows, int cols, int splits, int block, int& e,
                                            int& mt, int& nt, int& split) {
  const int at = place_of(block, N * rows * cols * splits);
  if (at < 0) return false;
  split = at % splits;
  const int tile = at / splits;
  e = tile / (rows * cols);
  banded(tile - e * rows * cols, rows, cols, mt, nt);
  return true;
}

// Most row tiles that R rows in N groups can make.
inline long max_row_tiles(int R, int N, int height) {
  return static_cast<long>(R) / height + (R < N ? R : N);
}

}  // namespace grp
}  // namespace moe
