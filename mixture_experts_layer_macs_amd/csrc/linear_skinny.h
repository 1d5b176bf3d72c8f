// y = x w^T for a few tokens (bf16): one workgroup per 16 weight rows (GLU: 8
// gate rows and their 8 up rows), 8 waves that take blocks of 64 k in turn.
// Operands go straight from memory to the registers of
// v_mfma_f32_16x16x32_bf16 (lane: row l % 16, k 8 (l / 16) .. + 7): a block is
// two loads of 16 rows x 64 bytes per operand fragment, the two halves of the
// same 128-byte lines.  The weights are read once; the RF fragments of 16
// tokens come from L2.  The waves' sums join through LDS in wave order.
//
// Bound by HBM for long weights and by one memory latency for short ones,
// which is why the panel is 16 rows wide (96 workgroups for a 1536 x 2048
// weight) and every load of a wave's first blocks is in flight at once.
// Measured: 1 token on a 1536 x 2048 weight 5.1 us, on 14336 x 4096 24 us
// (117 MB, 4.9 TB/s).
#pragma once

#include "common.h"
#include "linear_common.h"

namespace moe {
namespace lin {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct Skinny {
  const uint16_t *x, *w;
  int T, K, O;        // O: columns of y
  int panels, parts;  // weight panels, parts of the tokens
  Epilogue e;
};

constexpr int SK_WAVES = 8, SK_BLOCK = 64;

// Rows t0 .. of x (LISTED: of the stored rows in `token`) and columns n0 .. of y;
// red: the waves' sums.
template <int RF, bool GLU, bool LISTED>
__device__ __forceinline__ void skinny_tile(const Skinny& p, int n0, int t0, const int32_t* token,
                                            float (*red)[RF * 16][17]) {
  constexpr int NC = GLU ? 8 : 16;              // columns of y per workgroup
  constexpr int AHEAD = RF >= 4 ? 1 : 4 / RF;   // blocks in flight per wave
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
  const int r = lane & 15, k_lane = (lane >> 4) * 8;
  // rows past the end repeat the last one; their results are not stored
  const int wr = GLU ? (r < 8 ? min(n0 + r, p.O - 1) : p.O + min(n0 + r - 8, p.O - 1))
                     : min(n0 + r, p.O - 1);
  const uint16_t* w = p.w + static_cast<size_t>(wr) * p.K + k_lane;
  const uint16_t* x[RF];
#pragma unroll
  for (int f = 0; f < RF; ++f) {
    const int t = min(t0 + f * 16 + r, p.T - 1);
    x[f] = p.x + static_cast<size_t>(LISTED ? token[t] : t) * p.K + k_lane;
  }
  f32x4 acc[RF];
#pragma unroll
  for (int f = 0; f < RF; ++f) acc[f] = f32x4{0, 0, 0, 0};
  const int full = p.K / SK_BLOCK;
  int b = wave;
  for (; b + (AHEAD - 1) * SK_WAVES < full; b += AHEAD * SK_WAVES) {
    bf16x8 fw[AHEAD][2], fx[AHEAD][2][RF];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const size_t k = static_cast<size_t>(b + u * SK_WAVES) * SK_BLOCK + 32 * h;
        fw[u][h] = *reinterpret_cast<const bf16x8*>(w + k);
#pragma unroll
        for (int f = 0; f < RF; ++f) fx[u][h][f] = *reinterpret_cast<const bf16x8*>(x[f] + k);
      }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < RF; ++f)
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[u][h], fx[u][h][f], acc[f], 0, 0, 0);
  }
  for (; b * SK_BLOCK < p.K; b += SK_WAVES) {  // the rest, the last block cut at K
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = b * SK_BLOCK + 32 * h;
      const bool in = k + k_lane < p.K;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      const uint4 fw = in ? *reinterpret_cast<const uint4*>(w + k) : zero;
#pragma unroll
      for (int f = 0; f < RF; ++f) {
        const uint4 fx = in ? *reinterpret_cast<const uint4*>(x[f] + k) : zero;
        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8, fw), __builtin_bit_cast(bf16x8, fx), acc[f], 0, 0, 0);
      }
    }
  }
  // acc[f][i]: weight row 4 (l / 16) + i, token 16 f + l % 16
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][f * 16 + r][4 * (lane >> 4) + i] = acc[f][i];
  __syncthreads();
  constexpr int QUADS = NC / 4;
  for (int i = threadIdx.x; i < RF * 16 * QUADS; i += SK_WAVES * MOE_WAVE) {
    const int t = i / QUADS, c = i % QUADS * 4;
    if (t0 + t >= p.T || n0 + c >= p.O) continue;
    float g[4], u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      g[j] = u[j] = 0.f;
#pragma unroll
      for (int v = 0; v < SK_WAVES; ++v) {
        g[j] += red[v][t][c + j];
        if constexpr (GLU) u[j] += red[v][t][8 + c + j];
      }
    }
    finish<uint16_t, GLU, 4>(p.e, t0 + t, n0 + c, p.O, g, u);
  }
}

template <int RF, bool GLU>
__global__ __launch_bounds__(SK_WAVES* MOE_WAVE) void skinny_kernel(Skinny p) {
  __shared__ float red[SK_WAVES][RF * 16][17];
  const int total = p.panels * p.parts, per = (total + 7) / 8;
  const int id = blockIdx.x % 8 * per + blockIdx.x / 8;
  if (id >= total) return;
  skinny_tile<RF, GLU, false>(p, id / p.parts * (GLU ? 8 : 16), id % p.parts * RF * 16, nullptr, red);
}

}  // namespace lin
}  // namespace moe
