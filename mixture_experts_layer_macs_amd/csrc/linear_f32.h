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
  const int32_t* token;  // grouped products: stored rows of the gathered operand
};

// Which stored rows of an operand a product reads: as they lie, or those of a
// token list.
enum Gather { PLAIN, ROWS, COLUMNS };  // COLUMNS: of the column operand

template <bool LISTED>
__device__ __forceinline__ size_t stored(const int32_t* token, int i) {
  if constexpr (LISTED) return static_cast<size_t>(token[i]);
  else return static_cast<size_t>(i);
}

// Four values k, k + 1, .. of row m, zeros outside the matrix.
template <bool STRIDED, bool LISTED = false>
__device__ __forceinline__ f32x4 quad(const float* p, size_t ld, int m, int mend, int k, int kend,
                                      const int32_t* token = nullptr) {
  if constexpr (!STRIDED) {
    return m < mend && k < kend
               ? *reinterpret_cast<const f32x4*>(p + stored<LISTED>(token, m) * ld + k)
               : f32x4{0, 0, 0, 0};
  } else {
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = m < mend && k + i < kend ? p[stored<LISTED>(token, k + i) * ld + m] : 0.f;
    return v;
  }
}

// Small outputs: one 32 x 32 tile per workgroup, its four waves each a quarter
// of the reduction in turns of 8 k, operands straight from memory to the MFMA
// registers (lane: row l % 32; MFMA j of a turn takes k = j and j + 4), the
// waves' sums joined through LDS.  Bound by latency: with 64 workgroups a
// larger tile would leave the card empty.  256 x 128 -> 256: 4.2 us.
constexpr int SMALL_LDS = 4 * 32 * 33;  // floats per output matrix

template <bool RS, bool CS, bool GLU, Gather G = PLAIN>
__device__ __forceinline__ void f32_small_tile(const F32Prod& p, int bx, int by, float* lds) {
  constexpr int H = GLU ? 2 : 1, TURNS = 4;
  float(*red)[4][32][33] = reinterpret_cast<float(*)[4][32][33]>(lds);
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
  const int m0 = by * 32, n0 = bx * 32;
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
      a[u] = quad<RS, G == ROWS>(p.r, p.ldr, m, p.M, k, p.K, p.token);
#pragma unroll
      for (int h = 0; h < H; ++h)
        b[h][u] = quad<CS, G == COLUMNS>(p.c + h * static_cast<size_t>(p.N) * p.ldc, p.ldc, n, p.N, k,
                                         p.K, p.token);
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

template <bool RS, bool CS, bool GLU>
__global__ __launch_bounds__(256) void f32_small_kernel(F32Prod p) {
  __shared__ float lds[(GLU ? 2 : 1) * SMALL_LDS];
  f32_small_tile<RS, CS, GLU>(p, blockIdx.x, blockIdx.y, lds);
}

// Large outputs: tiles of 64 F x 64 F (F = 1 or 2), 4 waves of 32 F x 32 F,
// slices of 32 / F k through two LDS buffers laid out [k][m], the next two
// slices' loads in flight in registers while one is multiplied.  A slice is 16 F MFMAs
// of 64 cycles per wave, so the LDS traffic stays below the matrix pipe's time.
// 4096^3: 1.12 ms (123 TFLOP/s; the library 0.92 to 1.0).
template <bool STRIDED, bool MIX, int F, bool LISTED = false>
struct F32Stage {
  static constexpr int EXT = 64 * F, BK = 32 / F;
  static constexpr int PITCH = EXT + 4;  // floats: rows 4 banks apart, 16-byte aligned
  static constexpr int KQ = BK / 4, MQ = EXT / 4;
  f32x4 v[2];
  // Thread's share: contiguous: row t / KQ and 256 / KQ on, k quad t % KQ;
  // strided: k t / MQ and 256 / MQ on, m quad t % MQ.  MIX (gated weights):
  // every 32 rows are 16 gate rows and the 16 up rows of the same columns.
  __device__ __forceinline__ void fetch(const float* p, size_t ld, int valid, int k0, int kend,
                                        size_t up, const int32_t* token) {
    const int t = threadIdx.x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (!STRIDED) {
        const int row = t / KQ + 256 / KQ * i;
        const int at = MIX ? row / 32 * 16 + row % 16 : row;
        v[i] = quad<false, LISTED>(p + (MIX && row % 32 >= 16 ? up : 0), ld, at, valid,
                                   k0 + t % KQ * 4, kend, token);
      } else {
        const int k = k0 + t / MQ + 256 / MQ * i, m = t % MQ * 4;
        v[i] = k < kend && m < valid
                   ? *reinterpret_cast<const f32x4*>(p + stored<LISTED>(token, k) * ld + m)
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
        for (int j = 0; j < 4; ++j) s[(t % KQ * 4 + j) * PITCH + t / KQ + 256 / KQ * i] = v[i][j];
      } else {
        *reinterpret_cast<f32x4*>(s + (t / MQ + 256 / MQ * i) * PITCH + t % MQ * 4) = v[i];
      }
    }
  }
};

constexpr int LARGE_LDS = 2 * 32 * 68;  // floats of an operand's buffers: F = 2: 2 * 16 * 132

template <bool RS, bool CS, int F, bool GLU, bool PART, Gather G = PLAIN>
__device__ __forceinline__ void f32_large_tile(const F32Prod& p, int bx, int by, int bz, float* lds) {
  static_assert(!GLU || (!CS && !PART), "pairs of gate and up rows: y = x w^T only");
  typedef F32Stage<RS, false, F, G == ROWS> Row;
  typedef F32Stage<CS, GLU, F, G == COLUMNS> Col;
  constexpr int PITCH = Row::PITCH, BK = Row::BK, EXT = Row::EXT;
  static_assert(2 * BK * PITCH <= LARGE_LDS, "two buffers");
  float(*sr)[BK * PITCH] = reinterpret_cast<float(*)[BK * PITCH]>(lds);
  float(*sc)[BK * PITCH] = reinterpret_cast<float(*)[BK * PITCH]>(lds + LARGE_LDS);
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
  const int wm = wave / 2, wn = wave % 2;
  constexpr int NC = GLU ? EXT / 2 : EXT;
  const int m0 = by * EXT, n0 = bx * NC;
  const int k_lo = bz * p.per_split, k_hi = min(p.K, k_lo + p.per_split);
  const float* r = p.r + (RS ? m0 : G == ROWS ? 0 : m0 * p.ldr);
  const int32_t* token = p.token + (G == ROWS ? m0 : 0);
  const float* c = p.c + (CS ? n0 : n0 * p.ldc);
  const int mv = p.M - m0, nv = p.N - n0;
  Row row[2];
  Col col[2];
  auto fetch = [&](int set, int k0) {
    row[set].fetch(r, p.ldr, mv, k0, k_hi, 0, token);
    col[set].fetch(c, p.ldc, nv, k0, k_hi, GLU ? p.N * p.ldc : 0, token);
  };
  f32x16 acc[F][F];
#pragma unroll
  for (int x = 0; x < F; ++x)
#pragma unroll
    for (int y = 0; y < F; ++y)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[x][y][i] = 0.f;
  const int ml = wm * 32 * F + (lane & 31), nl = wn * 32 * F + (lane & 31), kl = lane >> 5;
  // Slices past the end fetch zeros without touching memory.
  fetch(0, k_lo);
  fetch(1, k_lo + BK);
  for (int k0 = k_lo; k0 < k_hi; k0 += 2 * BK) {
#pragma unroll
    for (int set = 0; set < 2; ++set) {
      if (set && k0 + BK >= k_hi) break;
      row[set].put(sr[set]);
      col[set].put(sc[set]);
      __syncthreads();
      fetch(set, k0 + (set + 2) * BK);
      const float *a = sr[set], *b = sc[set];
#pragma unroll
      for (int k = 0; k < BK; k += 2) {
        float fr[F], fc[F];
#pragma unroll
        for (int x = 0; x < F; ++x) fr[x] = a[(k + kl) * PITCH + ml + 32 * x];
#pragma unroll
        for (int y = 0; y < F; ++y) fc[y] = b[(k + kl) * PITCH + nl + 32 * y];
#pragma unroll
        for (int x = 0; x < F; ++x)
#pragma unroll
          for (int y = 0; y < F; ++y)
            acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x2f32(fc[y], fr[x], acc[x][y], 0, 0, 0);
      }
      // the buffer written next was last read before this slice's barrier
    }
  }
#pragma unroll
  for (int x = 0; x < F; ++x) {
    const int m = m0 + wm * 32 * F + 32 * x + (lane & 31);
    if (m >= p.M) continue;
#pragma unroll
    for (int y = 0; y < F; ++y)
#pragma unroll
      for (int q = 0; q < (GLU ? 2 : 4); ++q) {
        const int n = n0 + (wn * 32 * F + 32 * y) / (GLU ? 2 : 1) + 8 * q + 4 * kl;
        if (n >= p.N) continue;
        float g[4], u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] = acc[x][y][4 * q + i];
          if constexpr (GLU) u[i] = acc[x][y][4 * q + 8 + i];
        }
        if constexpr (PART)
          store4(p.part + (static_cast<size_t>(bz) * p.M + m) * p.N + n, g);
        else
          finish<float, GLU, 4>(p.e, m, n, p.N, g, u);
      }
  }
}

template <bool RS, bool CS, int F, bool GLU, bool PART>
__global__ __launch_bounds__(256) void f32_large_kernel(F32Prod p) {
  __shared__ __align__(16) float lds[2 * LARGE_LDS];
  f32_large_tile<RS, CS, F, GLU, PART>(p, blockIdx.x, blockIdx.y, blockIdx.z, lds);
}

}  // namespace lin
}  // namespace moe
