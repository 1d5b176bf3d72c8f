// bf16 grouped products on the dense layer's MFMA tiles (linear_mma.h): a
// workgroup finds its expert and tile from the expert offsets, points the
// operands at that expert's rows and weights, and runs mma_core.
//
//   FWD  y_r = act(W_e x_t)      rows of x, gathered, by W_e's rows
//   DX   dx_r = dz_r W_e         rows of dz by W_e's columns
//   DW   dW_e = sum dz_r x_t^T   reduction over the expert's rows, both operands
//                                reduction-strided, x laid out by rows beforehand
//
// Bound by the matrix pipe, by the partial tiles of ragged groups and by a tile's
// start and output (14 us beside 50 for 32 slices), which one workgroup a CU cannot
// hide.  Measured: 8192 tokens spread over 128 experts of 1536 x 2048, swiglu with z
// kept, 413 to 445 us (0.89 to 0.95 PFLOP/s); even groups of 512 rows 374; 8192 rows in
// 8 experts of 28672 x 4096 1675 to 1740 (1.11 to 1.15 PFLOP/s).
#pragma once

#include <type_traits>

#include "grouped_common.h"
#include "grouped_plan.h"
#include "linear_mma.h"
#include "linear_skinny.h"

namespace moe {
namespace grp {

using namespace lin;

constexpr int UNIT = 64;  // rows

struct Prod {
  const void *r, *c;     // FWD: x, w; DX: dz, w; DW: dz, x
  const int32_t* token;  // of the gathered operand (x); null: x holds the rows (DW in bf16: always)
  size_t x_rows;         // rows of x
  Groups g;
  int W, K;              // rows (GLU: gate and up) and columns of an expert's weights
  Epilogue e;            // y: dx, dw
  int splits;            // DW in parts: their number and [splits][N][W][K] sums
  float* part;
};

// The dense layer's row operand with the rows of a token list: the tile's rows
// are fixed, so the gather is in the lanes' offsets (x is at most 2^31 bytes).
template <int EXT, int SL>
struct GatherRows : Operand<false, false, EXT, lin::W, SL> {
  typedef Operand<false, false, EXT, lin::W, SL> Base;
  __device__ __forceinline__ void init_gather(const uint16_t* x, size_t ld, size_t x_rows,
                                              const int32_t* token, int valid, int wave, int lane) {
    const uint32_t row_bytes = static_cast<uint32_t>(ld) * 2;
    this->rsrc = buffer_rsrc(x, static_cast<uint32_t>(x_rows * row_bytes));
    const int lrow = lane / Base::CPR, slot = lane % Base::CPR;
#pragma unroll
    for (int q = 0; q < Base::Q; ++q) {
      const int row = (wave * Base::Q + q) * Base::RPL + lrow;
      const int ch = slot ^ Base::row_swizzle(row);
      if (q < 2) this->first[q] = ch * 8;
      this->voff[q] = row < valid ? static_cast<uint32_t>(token[row]) * row_bytes + ch * 16 : OOB_OFF;
    }
  }
};

// FWD, DX: one tile of at most BM rows.  An expert's rows are cut into units of
// 64 and these shared out evenly over its tiles, so that half a unit per expert
// is multiplied in vain, not half a tile.
template <int MODE, int BM, int BN, int SL, int RA, bool GLU, bool GATHER>
__device__ __forceinline__ void data_product(const Prod& p, int block, unsigned char* smem) {
  constexpr int NC = GLU ? BN / 2 : BN;
  constexpr bool STRIDED = MODE == DX;
  const int O = GLU ? p.W / 2 : p.W, N = MODE == FWD ? O : p.K, len = MODE == FWD ? p.K : p.W;
  const int cols = (N + NC - 1) / NC;
  int e, lo, hi, mt, nt;
  if (!data_tile(p.g, BM, cols, block, e, lo, hi, mt, nt)) return;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
  const int tiles = (hi - lo + BM - 1) / BM, units = (hi - lo + UNIT - 1) / UNIT;
  const int height = units / tiles + (mt < units % tiles);
  const int m0 = lo + (units / tiles * mt + min(mt, units % tiles)) * UNIT, n0 = nt * NC;
  const int rows = min(height * UNIT, hi - m0);
  const uint16_t* w = static_cast<const uint16_t*>(p.c) + static_cast<size_t>(e) * p.W * p.K;
  Operand<STRIDED, GLU, BN, lin::W, SL> col;
  col.init(w + (STRIDED ? n0 : n0 * static_cast<size_t>(p.K)), p.K, min(NC, N - n0), wave, lane,
           GLU ? O * static_cast<size_t>(p.K) : 0);
  auto run = [&](auto h) {
    constexpr int H = decltype(h)::value * UNIT;
    if constexpr (H <= BM) {
      GatherRows<H, SL> row;
      const uint16_t* r = static_cast<const uint16_t*>(p.r);
      if constexpr (GATHER)
        row.init_gather(r, len, p.x_rows, p.token + m0, rows, wave, lane);
      else
        row.init(r + static_cast<size_t>(m0) * len, len, rows, wave, lane);
      mma_core<false, STRIDED, H, BN, GLU, 8, SL, RA, SB, (RA * BM + SB * BN) * SL * 2>(
          row, col, 0, len, smem, [&](int r, int c, float* g, float* u) {
            if (r < rows && n0 + c < N) finish<uint16_t, GLU, 8>(p.e, m0 + r, n0 + c, N, g, u);
          });
    }
  };
  if (height == 1) run(std::integral_constant<int, 1>());
  else if (height == 2) run(std::integral_constant<int, 2>());
  else if (height == 3) run(std::integral_constant<int, 3>());
  else run(std::integral_constant<int, 4>());
}

// DW: one tile, or (PART) one of `splits` parts of its reduction.
template <int BM, int BN, int SL, int RA, bool PART>
__device__ __forceinline__ void weight_product(const Prod& p, int block, unsigned char* smem) {
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
  int e, mt, nt, split;
  if (!weight_tile(p.g.N, (p.W + BM - 1) / BM, (p.K + BN - 1) / BN, PART ? p.splits : 1, block, e, mt, nt,
                   split))
    return;
  const Span s = span_of(p.g, e);
  const int n0 = nt * BN, m0 = mt * BM, lo = s.lo, count = s.hi - s.lo;
  const int rows = min(BM, p.W - m0), width = min(BN, p.K - n0);
  int k_lo = 0, k_hi = count;
  if constexpr (PART) {
    const int per = ((count + p.splits - 1) / p.splits + SLICE - 1) / SLICE * SLICE;
    k_lo = uniform(split * per);
    k_hi = uniform(min(count, k_lo + per));
  }
  typedef std::conditional_t<PART, float, uint16_t> E;
  constexpr int V = PART ? 4 : 8;
  E* out = (PART ? reinterpret_cast<E*>(p.part) : static_cast<E*>(p.e.y)) +
           (PART ? static_cast<size_t>(split) * p.g.N + e : static_cast<size_t>(e)) * p.W * p.K;
  if (k_lo >= k_hi) {  // no rows: zeros
    for (int i = threadIdx.x; i < rows * (BN / V); i += lin::W * MOE_WAVE) {
      const int r = i / (BN / V), c = i % (BN / V) * V;
      if (c < width)
        *reinterpret_cast<u32x4*>(out + static_cast<size_t>(m0 + r) * p.K + n0 + c) = u32x4{0, 0, 0, 0};
    }
    return;
  }
  Operand<true, false, BM, lin::W, SL> row;
  row.init(static_cast<const uint16_t*>(p.r) + static_cast<size_t>(lo) * p.W + m0, p.W, rows, wave,
           lane);
  Operand<true, false, BN, lin::W, SL> col;
  col.init(static_cast<const uint16_t*>(p.c) + static_cast<size_t>(lo) * p.K + n0, p.K, width, wave,
           lane);
  mma_core<true, true, BM, BN, false, V, SL, RA>(
      row, col, k_lo, k_hi, smem, [&](int r, int c, float* g, float*) {
        if (r < rows && c < width) store_v<V>(out + static_cast<size_t>(m0 + r) * p.K + n0 + c, g);
      });
}

// RA: ring stages of the row operand.
// DW: GLU says that the reduction is in parts.
template <int MODE, int BM, int BN, int SL, int RA, int WGS, bool GLU, bool GATHER>
__global__ __launch_bounds__(lin::W* MOE_WAVE) __attribute__((amdgpu_waves_per_eu(WGS, WGS)))
void grouped_mma_kernel(Prod p) {
  extern __shared__ __align__(16) unsigned char smem[];
  if constexpr (MODE == DW) weight_product<BM, BN, SL, RA, GLU>(p, blockIdx.x, smem);
  else data_product<MODE, BM, BN, SL, RA, GLU, GATHER>(p, blockIdx.x, smem);
}

// FWD, a few rows to an expert: the dense layer's product for few tokens, 16 rows
// and 16 weight rows (8 gate and 8 up) to a workgroup, whose weights go straight
// to the MFMA registers.  Bound by HBM: one token, 8 experts of 1536 x 2048 (50 MB)
// 11.8 us, 4.3 TB/s.
template <bool GLU, bool GATHER>
__global__ __launch_bounds__(SK_WAVES* MOE_WAVE) void grouped_skinny_kernel(Prod p) {
  constexpr int NC = GLU ? 8 : 16;
  __shared__ float red[SK_WAVES][16][17];
  const int O = GLU ? p.W / 2 : p.W;
  int e, lo, hi, mt, nt;
  if (!data_tile(p.g, 16, (O + NC - 1) / NC, blockIdx.x, e, lo, hi, mt, nt)) return;
  Skinny q{};
  q.x = static_cast<const uint16_t*>(p.r) + (GATHER ? 0 : static_cast<size_t>(lo) * p.K);
  q.w = static_cast<const uint16_t*>(p.c) + static_cast<size_t>(e) * p.W * p.K;
  q.T = hi - lo;
  q.K = p.K;
  q.O = O;
  q.e = p.e;
  q.e.y = static_cast<uint16_t*>(p.e.y) + static_cast<size_t>(lo) * O;
  if (p.e.z) q.e.z = static_cast<uint16_t*>(p.e.z) + static_cast<size_t>(lo) * p.W;
  skinny_tile<1, GLU, GATHER>(q, nt * NC, mt * 16, GATHER ? p.token + lo : nullptr, red);
}

}  // namespace grp
}  // namespace moe
