// fp32 matrix products of the dense layer on v_mfma_f32_32x32x2_f32:
//   C[m][n] = sum_k R(m, k) C(n, k),
// each operand reduction-contiguous or reduction-strided as in linear_mma.h.
// The column operand is the MFMA's A, so a lane ends with groups of four
// consecutive output columns of one row.
#pragma once

#include "common.h"
#include "linear_common.h"

namespace moe {
namespace lin {

typedef float f32x16 __attribute__((ext_vector_type(16)));

struct F32Prod {
  const float *r, *c;
  size_t ldr, ldc;  // elements between their stored rows
  int M, N, K;      // output rows and columns (GLU: columns of y), reduction
  int per_split;    // reduction length of a split (large tiles)
  float* part;      // splits > 1: [splits][M][N] partial sums
  Epilogue e;
};

// Four values k, k + 1, .. of row m, zeros outside the matrix.
template <bool STRIDED>
__device__ __forceinline__ f32x4 quad(const float* p, size_t ld, int m, int mend, int k, int kend) {
  if constexpr (!STRIDED) {
    return m < mend && k < kend ? *reinterpret_cast<const f32x4*>(p + m * ld + k) : f32x4{0, 0, 0, 0};
  } else {
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = m < mend && k + i < kend ? p[(k + i) * ld + m] : 0.f;
    return v;
  }
}

// Small outputs: one 32 x 32 tile per workgroup, its four waves each a quarter
// of the reduction in turns of 8 k, operands straight from memory to the MFMA
// registers (lane: row l % 32; MFMA j of a turn takes k = j and j + 4), the
// waves' sums joined through LDS.  Bound by latency: with 64 workgroups a
// larger tile would leave the card empty.
template <bool RS, bool CS, bool GLU>
__global__ __launch_bounds__(256) void f32_small_kernel(F32Prod p) {
  constexpr int H = GLU ? 2 : 1, TURNS = 4;
  __shared__ float red[H][4][32][33];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
  const int m0 = blockIdx.y * 32, n0 = blockIdx.x * 32;
  const int m = m0 + (lane & 31), n = n0 + (lane & 31);
  f32x16 acc[H];
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[h][i] = 0.f;
  const int k_lane = wave * 8 + (lane >> 5) * 4;
  for (int k0 = 0; k0 < p.K; k0 += 32 * TURNS) {
    f32x4 a[TURNS], b[H][TURNS];
#pragma unroll
    for (int u = 0; u < TURNS; ++u) {
      const int k = k0 + 32 * u + k_lane;
      a[u] = quad<RS>(p.r, p.ldr, m, p.M, k, p.K);
#pragma unroll
      for (int h = 0; h < H; ++h)
        b[h][u] = quad<CS>(p.c + h * static_cast<size_t>(p.N) * p.ldc, p.ldc, n, p.N, k, p.K);
    }
#pragma unroll
    for (int u = 0; u < TURNS; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < H; ++h)
          acc[h] = __builtin_amdgcn_mfma_f32_32x32x2f32(b[h][u][j], a[u][j], acc[h], 0, 0, 0);
  }
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[h][wave][lane & 31][8 * q + 4 * (lane >> 5) + i] = acc[h][4 * q + i];
  __syncthreads();
  const int row = threadIdx.x / 8, col = threadIdx.x % 8 * 4;
  if (m0 + row >= p.M || n0 + col >= p.N) return;
  float v[2][4];
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[h][i] = (red[h][0][row][col + i] + red[h][1][row][col + i]) +
                (red[h][2][row][col + i] + red[h][3][row][col + i]);
  finish<float, GLU, 4>(p.e, m0 + row, n0 + col, p.N, v[0], v[1]);
}

// Large outputs: 128 x 128 tiles, 4 waves of 64 x 64, slices of 16 k through
// two LDS buffers laid out [k][m], the next slice's loads in flight in
// registers while one is multiplied.  A slice is 32 MFMAs of 64 cycles per
// wave, so the LDS traffic stays far below the matrix pipe's time.
template <bool STRIDED>
struct F32Stage {
  static constexpr int PITCH = 132;  // floats: rows 4 banks apart, 16-byte aligned
  f32x4 v[2];
  // thread's share: contiguous: rows t / 4 and + 64, k quad t % 4; strided:
  // k t / 32 and + 8, m quad t % 32
  __device__ __forceinline__ void fetch(const float* p, size_t ld, int valid, int k0, int kend) {
    const int t = threadIdx.x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (!STRIDED) {
        v[i] = quad<false>(p, ld, t / 4 + 64 * i, valid, k0 + t % 4 * 4, kend);
      } else {
        const int k = k0 + t / 32 + 8 * i, m = t % 32 * 4;
        v[i] = k < kend && m < valid ? *reinterpret_cast<const f32x4*>(p + k * ld + m)
                                     : f32x4{0, 0, 0, 0};
      }
    }
  }
  __device__ __forceinline__ void put(float* s) const {
    const int t = threadIdx.x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (!STRIDED) {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[(t % 4 * 4 + j) * PITCH + t / 4 + 64 * i] = v[i][j];
      } else {
        *reinterpret_cast<f32x4*>(s + (t / 32 + 8 * i) * PITCH + t % 32 * 4) = v[i];
      }
    }
  }
};

template <bool RS, bool CS, bool GLU, bool PART>
__global__ __launch_bounds__(256) void f32_large_kernel(F32Prod p) {
  static_assert(!GLU || (!CS && !PART), "pairs of gate and up rows: y = x w^T only");
  constexpr int PITCH = F32Stage<false>::PITCH, BK = 16;
  __shared__ __align__(16) float sr[2][BK * PITCH], sc[2][BK * PITCH];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
  const int wm = wave / 2, wn = wave % 2;
  constexpr int NC = GLU ? 64 : 128;
  const int m0 = blockIdx.y * 128, n0 = blockIdx.x * NC;
  const int k_lo = blockIdx.z * p.per_split, k_hi = min(p.K, k_lo + p.per_split);
  const float* r = p.r + (RS ? m0 : m0 * p.ldr);
  const float* c = p.c + (CS ? n0 : n0 * p.ldc);
  const int mv = p.M - m0, nv = p.N - n0;
  F32Stage<RS> row;
  F32Stage<CS> col;
  auto fetch = [&](int k0) {
    row.fetch(r, p.ldr, mv, k0, k_hi);
    if constexpr (GLU) {  // tile rows 0 .. 63 gate, 64 .. 127 up
      const int t = threadIdx.x;
      col.v[0] = quad<false>(c, p.ldc, t / 4, nv, k0 + t % 4 * 4, k_hi);
      col.v[1] = quad<false>(c + static_cast<size_t>(p.N) * p.ldc, p.ldc, t / 4, nv,
                             k0 + t % 4 * 4, k_hi);
    } else {
      col.fetch(c, p.ldc, nv, k0, k_hi);
    }
  };
  f32x16 acc[2][2];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[x][y][i] = 0.f;
  const int ml = wm * 64 + (lane & 31), kl = lane >> 5;
  // GLU: a wave's two column fragments are 32 gate columns and their up columns
  const int nl = (GLU ? wn * 32 : wn * 64) + (lane & 31);
  constexpr int YSTEP = GLU ? 64 : 32;
  fetch(k_lo);
  int buf = 0;
  for (int k0 = k_lo; k0 < k_hi; k0 += BK, buf ^= 1) {
    row.put(sr[buf]);
    col.put(sc[buf]);
    __syncthreads();
    if (k0 + BK < k_hi) fetch(k0 + BK);
    const float *a = sr[buf], *b = sc[buf];
#pragma unroll
    for (int k = 0; k < BK; k += 2) {
      float fr[2], fc[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) fr[x] = a[(k + kl) * PITCH + ml + 32 * x];
#pragma unroll
      for (int y = 0; y < 2; ++y) fc[y] = b[(k + kl) * PITCH + nl + YSTEP * y];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x2f32(fc[y], fr[x], acc[x][y], 0, 0, 0);
    }
    // the buffer written next was last read before this iteration's barrier
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int m = m0 + wm * 64 + 32 * x + (lane & 31);
    if (m >= p.M) continue;
#pragma unroll
    for (int y = 0; y < (GLU ? 1 : 2); ++y)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + (GLU ? wn * 32 : wn * 64 + 32 * y) + 8 * q + 4 * kl;
        if (n >= p.N) continue;
        float g[4], u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] = acc[x][y][4 * q + i];
          if constexpr (GLU) u[i] = acc[x][1][4 * q + i];
        }
        if constexpr (PART)
          store4(p.part + (static_cast<size_t>(blockIdx.z) * p.M + m) * p.N + n, g);
        else
          finish<float, GLU, 4>(p.e, m, n, p.N, g, u);
      }
  }
}

}  // namespace lin
}  // namespace moe
