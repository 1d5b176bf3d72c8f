// fp32 grouped products on the dense layer's tiles (linear_f32.h): a workgroup
// finds its expert and tile and hands that expert's rows and weights to the
// dense tile as a product of its own.
#pragma once

#include "grouped_common.h"
#include "grouped_mma.h"
#include "linear_f32.h"

namespace moe {
namespace grp {

// EDGE: 32, 64 or 128, the tile's edge (GLU: half as many columns for 64 and 128).
template <int MODE, bool GLU, bool GATHER, int EDGE>
__device__ __forceinline__ void f32_tile(const Prod& p, int block, float* lds) {
  constexpr Gather G = !GATHER ? PLAIN : MODE == DW ? COLUMNS : ROWS;
  constexpr int NC = GLU && EDGE > 32 ? EDGE / 2 : EDGE;
  const float *R = static_cast<const float*>(p.r), *C = static_cast<const float*>(p.c);
  const int O = GLU ? p.W / 2 : p.W, N = MODE == FWD ? O : p.K;
  const int cols = (N + NC - 1) / NC;
  int e, lo, hi, mt, nt;
  if constexpr (MODE == DW) {
    const int rows = (p.W + EDGE - 1) / EDGE;
    if (block >= p.g.N * rows * cols) return;
    e = block / (rows * cols);
    banded(block - e * rows * cols, rows, cols, mt, nt);
    const Span s = span_of(p.g, e);
    lo = s.lo;
    hi = s.hi;
  } else {
    if (!data_tile(p.g, EDGE, cols, block, e, lo, hi, mt, nt)) return;
  }
  const size_t weights = static_cast<size_t>(e) * p.W * p.K;
  F32Prod q{};
  q.N = N;
  q.e = p.e;
  q.ldc = p.K;
  if constexpr (MODE == DW) {  // no rows: a reduction of no length, zeros
    q.r = R + static_cast<size_t>(lo) * p.W;
    q.ldr = p.W;
    q.c = C + (GATHER ? 0 : static_cast<size_t>(lo) * p.K);
    q.M = p.W;
    q.K = hi - lo;
    q.e.y = static_cast<float*>(p.e.y) + weights;
  } else {
    const int len = MODE == FWD ? p.K : p.W;
    q.r = R + (GATHER ? 0 : static_cast<size_t>(lo) * len);
    q.ldr = len;
    q.c = C + weights;
    q.M = hi - lo;
    q.K = len;
    q.e.y = static_cast<float*>(p.e.y) + static_cast<size_t>(lo) * N;
    if (p.e.z) q.e.z = static_cast<float*>(p.e.z) + static_cast<size_t>(lo) * p.W;
  }
  if constexpr (GATHER) q.token = p.token + lo;
  q.per_split = q.K;
  constexpr bool RS = MODE == DW, CS = MODE != FWD;
  if constexpr (EDGE == 32) f32_small_tile<RS, CS, GLU, G>(q, nt, mt, lds);
  else f32_large_tile<RS, CS, EDGE / 64, GLU, false, G>(q, nt, mt, 0, lds);
}

constexpr int f32_lds(bool glu, int edge) {
  return edge == 32 ? (glu ? 2 : 1) * SMALL_LDS : 2 * LARGE_LDS;
}

template <int MODE, bool GLU, bool GATHER, int EDGE>
__global__ __launch_bounds__(256) void grouped_f32_kernel(Prod p, int tiles) {
  __shared__ __align__(16) float lds[f32_lds(GLU, EDGE)];
  for (int at = blockIdx.x; at < tiles; at += gridDim.x) {
    f32_tile<MODE, GLU, GATHER, EDGE>(p, at, lds);
    __syncthreads();
  }
}

// Both products of a small backward pass in one launch; workgroups from dw0 on are dw's.
template <bool GATHER>
__global__ __launch_bounds__(256) void grouped_f32_pair_kernel(Prod dx, Prod dw, int dw0) {
  __shared__ __align__(16) float lds[f32_lds(false, 32)];
  const int block = blockIdx.x;
  if (block < dw0) f32_tile<DX, false, false, 32>(dx, block, lds);
  else f32_tile<DW, false, GATHER, 32>(dw, block - dw0, lds);
}

}  // namespace grp
}  // namespace moe
