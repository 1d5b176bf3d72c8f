// Which kernels a call of the dense layer runs, and what its workspace holds:
// functions of the sizes, the type and the number of compute units, without
// device code (the tests compile this file for the host and look at the choice
// of every tested size).
#pragma once

#include <stddef.h>

#include <algorithm>
#include <cmath>

#include "../../include/moe_macs.h"

namespace moe {
namespace lin {

struct Plan {
  int tile;    // index into TILES (bf16), edge of the tile (fp32)
  int splits;  // of the reduction
  double us;   // estimate
};

struct Tile {
  int m, n;
};
constexpr Tile TILES[] = {{256, 256}, {256, 192}, {192, 256}, {128, 128}};

// Tile and splits of a bf16 product of M x W outputs: the least time by a
// model fitted to 4 tiles and up to 16 splits of 50 shapes of all four operand
// layouts (136 .. 8192 rows, 64 .. 14336 columns, reductions of 64 .. 8192; 9 %
// rms off, its choice 1.5 % above the best of each shape in the mean).  Times
// in us.  Large tiles take a CU each, in rounds: 1.25 per slice of a 256 x 256
// tile and 10.1 for its output, in proportion to the area, and 2.3 to start;
// 128 x 128 tiles, up to two on a CU at once, 0.43 per slice and 2.0 for the
// output each.  Partial sums cost a launch and their traffic; the column
// operand streams at 4.5 TB/s at best.
inline Plan plan(int M, int W, int K, int cus) {
  Plan best{3, 1, 1e30};
  for (int t = 0; t < 4; ++t) {
    const long tiles = static_cast<long>((M + TILES[t].m - 1) / TILES[t].m) *
                       ((W + TILES[t].n - 1) / TILES[t].n);
    const double area = TILES[t].m * TILES[t].n / 65536.0;
    for (int want = 1; want <= 8; ++want) {
      const int per = ((K + want - 1) / want + 63) / 64, splits = (K + per * 64 - 1) / (per * 64);
      if (splits != want) continue;
      const double rounds = static_cast<double>((tiles * splits + cus - 1) / cus);
      const double out = splits > 1 ? 0.65 : 1.0;  // partial sums are stored as they are
      double us = t < 3 ? rounds * (per * 1.25 * area + 10.1 * area * out + 2.3) + 1.0
                        : rounds * (per * 0.43 + 2.0 * out) + 3.3;
      us = std::max(us, static_cast<double>(W) * K * (2 / 4.5e6));
      if (splits > 1) us += 3.3 + splits * (0.4 + static_cast<double>(M) * W * (4 / 3.9e6));
      if (us < best.us) best = Plan{t, splits, us};
    }
  }
  return best;
}

// The same for fp32, from a sweep of 12 shapes in three layouts: a 32 x 32 tile
// takes 0.009 us per k (0.011 with a strided operand), a 64 x 64 tile 0.028
// alone on its CU and 0.025 with others, a 128 x 128 tile 0.084 and 0.068, on
// top of about 3 us; splits as above.  1024^3: 31 us with 64 x 64 tiles, 41
// with 32 x 32, 34 with 128 x 128 in four splits; 512^3: 7.3, 10.3 and 15.4.
inline Plan plan_f32(int M, int W, int K, bool strided, int cus) {
  Plan best{32, 1, 1e30};
  for (int tile = 32; tile <= 128; tile *= 2) {
    const double tiles = static_cast<double>((M + tile - 1) / tile) * ((W + tile - 1) / tile);
    for (int want = 1; want <= (tile == 32 ? 1 : 8); ++want) {
      const int per = ((K + want - 1) / want + 31) / 32 * 32, splits = (K + per - 1) / per;
      if (splits != want) continue;
      double load = tiles * splits / cus;
      if (load <= 4) load = std::ceil(load);  // the fullest CU sets the time
      const double alone = tile == 32 ? (strided ? 0.011 : 0.009) : tile == 64 ? 0.028 : 0.084;
      const double shared = tile == 32 ? alone : tile == 64 ? 0.025 : 0.068;
      double us = 2.8 + std::min(K, per) * std::max(alone, load * shared);
      if (splits > 1) us += 3.5 + static_cast<double>(splits) * M * W * (4 / 4.0e6);
      if (us < best.us) best = Plan{tile, splits, us};
    }
  }
  return best;
}

// Few tokens: the skinny product or the tiles, whichever is estimated faster.
// The skinny one is bound by its loads' addresses: a block of 64 k costs a
// workgroup 0.25 us for the weights and 0.4 us for each 16 tokens (less for
// rows that repeat), on top of 3 us, and the weights stream at 5.5 TB/s at
// best (sweep of 7 weights of 256 x 4096 .. 14336 x 4096, 1 .. 512 tokens).
// 768 x 2048: 3.9 us for 1 token, 6.1 for 128 (tiles: 9.6); 4096 x 14336: 24
// for 1 token, but 145 for 128, where two splits of 128 x 128 tiles take 36.
// least: the tiles' estimate.  Returns the fragments of 16 tokens per
// workgroup; 0: tiles.
inline int skinny_plan(int T, int K, int W, double least, int cus) {
  int best = 0;
  if (T > 128) return best;
  for (int rf = 1; rf <= 8; rf *= 2) {
    if (rf > 1 && T <= rf * 8) break;  // half the fragments would be empty
    const double wgs = static_cast<double>((W + 15) / 16) * ((T + rf * 16 - 1) / (rf * 16));
    const double turns = std::max(1.0, wgs / cus) * K / 512.0;
    const double full = 0.25 + 0.75 * std::min(1.0, T / (16.0 * rf));
    const double us = 3.0 + std::max(turns * 0.25, static_cast<double>(W) * K * (2 / 5.5e6)) +
                      turns * 0.4 * rf * full;
    if (us < least) {
      least = us;
      best = rf;
    }
  }
  return best;
}

// --------------------------------------------------------------- workspaces
inline size_t elem_size(int dtype) { return dtype == MOE_BF16 ? 2 : 4; }
inline size_t up256(size_t n) { return (n + 255) & ~size_t(255); }
inline int width(int O, int act) { return act == MOE_ACT_SWIGLU ? 2 * O : O; }

constexpr int ROWT = 8;  // rows of an activation-gradient block side by side

struct BackPlan {
  int rows, blocks;   // token rows of an act_grad block, their number
  Plan x, w;          // dx, dw
  bool pair;          // both products in one launch
  size_t sums, part_x, part_w, bytes;  // offsets (dz at 0), size
};

inline size_t part_bytes(const Plan& p, int M, int W) {
  return p.splits > 1 ? up256(static_cast<size_t>(p.splits) * M * W * 4) : 0;
}

struct ForwardPlan {
  Plan p;
  int rf;  // of the skinny product; 0: tiles
  size_t bytes;
};

inline ForwardPlan forward_plan(int T, int K, int O, int act, int dtype, int cus) {
  ForwardPlan f{Plan{}, 0, 256};
  if (T == 0) return f;
  const int W = width(O, act);
  if (dtype == MOE_BF16) {
    f.p = plan(T, W, K, cus);
    f.rf = skinny_plan(T, K, W, f.p.us, cus);
  } else {
    f.p = plan_f32(T, W, K, false, cus);
  }
  if (!f.rf) f.bytes += part_bytes(f.p, T, W);
  return f;
}

inline BackPlan back_plan(int T, int K, int O, int act, int dtype, int cus) {
  BackPlan p{};
  const int W = width(O, act);
  p.rows = std::max(ROWT, (T + 255) / 256);
  p.blocks = (T + p.rows - 1) / p.rows;
  p.sums = act == MOE_ACT_NONE ? 0 : up256(static_cast<size_t>(T) * W * elem_size(dtype));
  p.part_x = p.sums + up256(static_cast<size_t>(p.blocks) * W * 4);
  p.part_w = p.part_x;
  p.bytes = p.part_x + 256;
  if (T == 0) return p;
  const bool bf16 = dtype == MOE_BF16;
  p.x = bf16 ? plan(T, K, W, cus) : plan_f32(T, K, W, true, cus);
  p.w = bf16 ? plan(W, K, T, cus) : plan_f32(W, K, T, true, cus);
  p.pair = p.x.tile == p.w.tile && p.x.tile == (bf16 ? 3 : 32);
  const size_t bx = part_bytes(p.x, T, K), bw = part_bytes(p.w, W, K);
  if (p.pair) p.part_w += bx;  // side by side; one after the other otherwise
  p.bytes += p.pair ? bx + bw : std::max(bx, bw);
  return p;
}

}  // namespace lin
}  // namespace moe
