// Which kernel a grouped product runs: functions of the sizes and the number of
// compute units, without device code (the tests compile this file for the host).
// The rows of each expert are known on the device only, so the choice goes by
// their mean.
#pragma once

#include <algorithm>
#include <cmath>

namespace moe {
namespace grp {

enum { FWD, DX, DW };

// Tiles of the bf16 products
enum { TILE_256, TILE_128, TILE_128x256, STREAM, SKINNY };

constexpr int STREAM_EXPERTS = 512;  // most that the streaming kernel's plan holds

inline double rounds(double tiles, int cus) { return std::ceil(tiles / cus); }

// A weight gradient of few tiles over many rows: its reduction in `splits` parts,
// whose fp32 sums a second launch adds; the time with 128 x 128 tiles. In parts and
// whole, us: one expert of 512^2 with 8192 rows 17.5 and 61.8, two of 1024^2 with 8192
// each 48 and 67, four of 768^2 with 8192 each 54 and 67.
inline double split_us(int R, int N, int W, int K, int splits, int cus) {
  const double tiles = N * std::ceil(W / 128.0) * std::ceil(K / 128.0);
  const double slices = static_cast<double>(R) / std::min(N, R) / 64 / splits;
  const double join = splits > 1 ? 4 + splits * (static_cast<double>(N) * W * K / 1.0e6) : 0;
  return rounds(tiles * splits, cus) * (slices * 0.57 + 2) + 4 + join;
}
inline int split_choice(int R, int N, int W, int K, int cus) {
  int best = 1;
  for (int s = 2; s <= 8; ++s)
    if (split_us(R, N, W, K, s, cus) < split_us(R, N, W, K, best, cus)) best = s;
  return best;
}

// rows, W, K: of a product as in Prod (FWD with a gated activation: gate and up).
// Times in us, from sweeps of 64 .. 1024 rows per expert, 128 experts, weights of
// 512^2 .. 4096^2: a slice of 64 k takes a 256 x 256 tile 1.55 (the matrix pipe at
// its power limit) on top of 14 (10 for a weight gradient), a 128 x 128 tile, two to
// a CU, 0.57 on top of 2.  128 experts of 1536 x 2048:
//   64 rows   dx 165 with 256 x 256 tiles, 170 with 128 x 128, and 150 with 128 x
//             256 and slices of 32: it is the weights that are read, 5.4 TB/s, by
//             two workgroups a CU
//             dw 200 streaming, 250 with 256 x 256 tiles, 274 with 128 x 128
//   512 rows  dx 395 streaming, 432, 523 and 481; dw 470, 530, 642; forward 374 and 429
// Few rows: where the 128 x 128 tiles leave half the compute units without one, 16
// weight rows to a workgroup: 8 experts with a row each 11.8 us, 16.1 with tiles
// (768 x 2048 swiglu); 16 such experts 20.3 and 18.8, 2048 x 768 10.0 and 8.9.
// The streaming kernel deals whole experts to the XCDs, which takes several
// for each: with 8 experts it took 1.7 times as long as the tiles, with 128 less than
// they did (above).  Between those the border at 64 is not measured.  That a few of
// many experts hold the rows does not show in the mean, and costs (grouped_stream.h).
inline int tile_choice(int mode, int R, int N, int W, int K, int cus) {
  const int used = std::min(N, R);  // experts that can have rows
  const double rows = static_cast<double>(R) / used;
  auto tiles = [&](int m, int n) {
    const double a = std::ceil((mode == DW ? W : rows) / m);
    const double b = std::ceil(static_cast<double>(mode == FWD ? W : K) / n);
    return (mode == DW ? N : used) * a * b;
  };
  if (mode == DW && N >= 64 && N <= STREAM_EXPERTS && W > 128 && K > 128) return STREAM;
  if (mode == FWD && rows <= 16 && K >= 1024 && tiles(128, 128) * 2 < cus) return SKINNY;
  if (mode == DX && rows <= 128 && tiles(128, 256) >= cus) return TILE_128x256;
  const double slices = (mode == DW ? rows : mode == FWD ? K : W) / 64.0;
  const double height = mode == DW ? 1.0 : std::min(1.0, std::ceil(rows / 64) / 4);
  const double large = rounds(tiles(256, 256), cus) *
                       (slices * std::max(0.4, 1.55 * height) + (mode == DW ? 10 : 14));
  double small = rounds(tiles(128, 128), cus) * (slices * 0.57 + 2) + 4;
  if (mode == DW) small = std::min(small, split_us(R, N, W, K, split_choice(R, N, W, K, cus), cus));
  if (mode == DX && large <= small && N >= 64 && N <= STREAM_EXPERTS) return STREAM;
  return large <= small ? TILE_256 : TILE_128;
}

// The same for fp32: the edge of the tile, by the dense layer's measures (us per
// k of a tile alone on its compute unit, and with others).
//   512^3 in one expert: see plan_f32, whose model this is without splits
inline int tile_choice_f32(int mode, int R, int N, int W, int K, int cus) {
  const int used = std::min(N, R);
  const double rows = static_cast<double>(R) / used;
  int best = 32;
  double least = 1e30;
  for (int edge = 32; edge <= 128; edge *= 2) {
    const double a = std::ceil((mode == DW ? W : rows) / edge);
    const double b = std::ceil(static_cast<double>(mode == FWD ? W : K) / edge);
    const double len = mode == DW ? rows : mode == FWD ? K : W;
    double load = (mode == DW ? N : used) * a * b / cus;
    if (load <= 4) load = std::ceil(load);
    const double alone = edge == 32 ? (mode == FWD ? 0.009 : 0.011) : edge == 64 ? 0.028 : 0.084;
    const double shared = edge == 32 ? alone : edge == 64 ? 0.025 : 0.068;
    const double us = len * std::max(alone, load * shared);
    if (us < least) {
      least = us;
      best = edge;
    }
  }
  return best;
}

}  // namespace grp
}  // namespace moe
