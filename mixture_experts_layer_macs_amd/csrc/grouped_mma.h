// bf16 grouped products on the dense layer's MFMA tiles (linear_mma.h): a
// workgroup finds its expert and tile from the expert offsets, points the
// operands at that expert's rows and weights, and runs mma_core.
//
//   FWD  y_r = act(W_e x_t)      rows of x, gathered, by W_e's rows
//   DX   dx_r = dz_r W_e         rows of dz by W_e's columns
//   DW   dW_e = sum dz_r x_t^T   reduction over the expert's rows, both operands
//                                reduction-strided, x gathered along it
#pragma once

#include "grouped_common.h"
#include "linear_mma.h"

namespace moe {
namespace grp {

using namespace lin;

enum { FWD, DX, DW };

struct Prod {
  const void *r, *c;     // FWD: x, w; DX: dz, w; DW: dz, x
  const int32_t* token;  // of the gathered operand (x); null: x holds the rows
  size_t x_rows;         // rows of x
  Groups g;
  int W, K;              // rows (GLU: gate and up) and columns of an expert's weights
  Epilogue e;            // y: dx, dw
};

// The dense layer's row operand with the rows of a token list: the tile's rows
// are fixed, so the gather is in the lanes' offsets (x is at most 2^31 bytes).
template <int EXT>
struct GatherRows : Operand<false, false, EXT, lin::W> {
  typedef Operand<false, false, EXT, lin::W> Base;
  __device__ __forceinline__ void init_gather(const uint16_t* x, size_t ld, size_t x_rows,
                                              const int32_t* token, int valid, int wave, int lane) {
    const uint32_t row_bytes = static_cast<uint32_t>(ld) * 2;
    this->rsrc = buffer_rsrc(x, static_cast<uint32_t>(x_rows * row_bytes));
    const int lrow = lane / 8, slot = lane % 8;
#pragma unroll
    for (int q = 0; q < Base::Q; ++q) {
      const int row = (wave * Base::Q + q) * 8 + lrow;
      const int ch = slot ^ Base::row_swizzle(row);
      if (q < 2) this->first[q] = ch * 8;
      this->voff[q] = row < valid ? static_cast<uint32_t>(token[row]) * row_bytes + ch * 16 : OOB_OFF;
    }
  }
};

// The reduction-strided operand whose k are the rows of a token list.  A wave's
// loads of a slice are 16 consecutive k, whose tokens it holds in scalar
// registers: fetch requests them a slice ahead, prepare, behind a wait that the
// loop makes anyway, turns them into the lanes' offsets.
template <int EXT>
struct GatherStrided {
  typedef Operand<true, false, EXT, lin::W> Base;
  static constexpr int BYTES = Base::BYTES, Q = Base::Q, CPR = EXT / 8, PER = 64 / CPR;
  static_assert(64 % CPR == 0 && PER * Q == 16 && lin::W * 16 == SLICE, "16 rows per wave and slice");
  typedef __attribute__((address_space(4))) const int32_t scalar_i32;
  i32x4 rsrc;
  uint32_t voff[Q], step, ch;
  const int32_t* token;
  int left, sub;  // entries of the token list, the lane's row of a load's PER
  bool live;
  int32_t t[16];
  int at;         // k of t[0]

  __device__ __forceinline__ void init(const uint16_t* x, int n0, size_t ld, size_t x_rows,
                                       const int32_t* tok, int tokens, int valid, int wave, int lane) {
    step = static_cast<uint32_t>(ld) * 2;
    rsrc = buffer_rsrc(x, static_cast<uint32_t>(x_rows * step));
    token = tok;
    left = tokens;
    sub = lane / CPR;
    // row of a load: PER (16 wave + ..) + sub; PER is a multiple of 2, so the swizzle depends on q and sub
    ch = static_cast<uint32_t>(lane % CPR);
    n_bytes = static_cast<uint32_t>(n0) * 2;
    valid_ch = valid / 8;
  }
  uint32_t n_bytes;
  int valid_ch;
  __device__ __forceinline__ void fetch(int k0, int wave) {
    at = k0 + wave * 16;
    scalar_i32* p = (scalar_i32*)(token);
    if (at + 16 <= left) {
#pragma unroll
      for (int i = 0; i < 16; ++i) t[i] = p[at + i];
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) t[i] = p[min(at + i, left - 1)];
    }
  }
  __device__ __forceinline__ void prepare(int, int kend) {
    uint32_t off[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      off[i] = at + i < kend ? static_cast<uint32_t>(t[i]) * step + n_bytes : OOB_OFF;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      uint32_t v = off[q * PER];
#pragma unroll
      for (int s = 1; s < PER; ++s) v = sub == s ? off[q * PER + s] : v;
      const uint32_t c = ch ^ static_cast<uint32_t>(Base::swizzle(q * PER + sub));
      voff[q] = static_cast<int>(c) < valid_ch ? v + c * 16 : OOB_OFF;
    }
  }
  __device__ __forceinline__ void load(int q, int, int, uint32_t lds, int wave) const {
    lds_dma16(rsrc, voff[q], 0, lds + (wave * Q + q) * 1024);
  }
};

template <int MODE, int BM, int BN, bool GLU, bool GATHER>
__device__ __forceinline__ void grouped_tile(const Prod& p, int block, unsigned char* smem) {
  const uint16_t *R = static_cast<const uint16_t*>(p.r), *C = static_cast<const uint16_t*>(p.c);
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
  constexpr int NC = GLU ? BN / 2 : BN;
  const int O = GLU ? p.W / 2 : p.W, N = MODE == FWD ? O : p.K;
  const int cols = (N + NC - 1) / NC;
  int e, lo, hi, mt, nt;
  if constexpr (MODE == DW) {
    const int rows = (p.W + BM - 1) / BM;
    if (!weight_tile(p.g.N, rows, cols, block, e, mt, nt)) return;
    const Span s = span_of(p.g, e);
    lo = s.lo;
    hi = s.hi;
  } else {
    if (!data_tile(p.g, BM, cols, block, e, lo, hi, mt, nt)) return;
  }
  const int n0 = nt * NC, m0 = mt * BM;
  if constexpr (MODE == DW) {
    uint16_t* out = static_cast<uint16_t*>(p.e.y) + static_cast<size_t>(e) * p.W * p.K;
    const int rows = min(BM, p.W - m0), width = min(BN, N - n0);
    if (lo == hi) {  // no rows: zeros
      for (int i = threadIdx.x; i < rows * (BN / 8); i += lin::W * MOE_WAVE) {
        const int r = i / (BN / 8), c = i % (BN / 8) * 8;
        if (c < width)
          *reinterpret_cast<u32x4*>(out + static_cast<size_t>(m0 + r) * p.K + n0 + c) = u32x4{0, 0, 0, 0};
      }
      return;
    }
    Operand<true, false, BM, lin::W> row;
    row.init(R + static_cast<size_t>(lo) * p.W + m0, p.W, rows, wave, lane);
    auto chunk = [&](int r, int c, float* g, float*) {
      if (r < rows && c < width) store_v<8>(out + static_cast<size_t>(m0 + r) * p.K + n0 + c, g);
    };
    if constexpr (GATHER) {
      GatherStrided<BN> col;
      col.init(C, n0, p.K, p.x_rows, p.token + lo, p.g.R - lo, width, wave, lane);
      mma_core<true, true, BM, BN, false, 8>(row, col, 0, hi - lo, smem, chunk);
    } else {
      Operand<true, false, BN, lin::W> col;
      col.init(C + static_cast<size_t>(lo) * p.K + n0, p.K, width, wave, lane);
      mma_core<true, true, BM, BN, false, 8>(row, col, 0, hi - lo, smem, chunk);
    }
  } else {
    const int m1 = lo + m0, rows = min(BM, hi - m1);
    const int len = MODE == FWD ? p.K : p.W;
    GatherRows<BM> row;
    if constexpr (GATHER)
      row.init_gather(R, len, p.x_rows, p.token + m1, rows, wave, lane);
    else
      row.init(R + static_cast<size_t>(m1) * len, len, rows, wave, lane);
    const uint16_t* w = C + static_cast<size_t>(e) * p.W * p.K;
    constexpr bool STRIDED = MODE == DX;
    Operand<STRIDED, GLU, BN, lin::W> col;
    col.init(w + (STRIDED ? n0 : n0 * static_cast<size_t>(p.K)), p.K, min(NC, N - n0), wave, lane,
             GLU ? O * static_cast<size_t>(p.K) : 0);
    mma_core<false, STRIDED, BM, BN, GLU, 8>(
        row, col, 0, len, smem, [&](int r, int c, float* g, float* u) {
          if (r < rows && n0 + c < N) finish<uint16_t, GLU, 8>(p.e, m1 + r, n0 + c, N, g, u);
        });
  }
}

template <int MODE, int BM, int BN, int WGS, bool GLU, bool GATHER>
__global__ __launch_bounds__(lin::W* MOE_WAVE) __attribute__((amdgpu_waves_per_eu(WGS, WGS)))
void grouped_mma_kernel(Prod p) {
  extern __shared__ __align__(16) unsigned char smem[];
  grouped_tile<MODE, BM, BN, GLU, GATHER>(p, blockIdx.x, smem);
}

}  // namespace grp
}  // namespace moe
