// moe_grouped_linear and moe_grouped_linear_backward: the routed experts'
// products over ragged groups of rows, and their gradients.
//
//   z_r = W_e x_t,  y_r = act(z_r);   dz = dy act'(z)
//   dx_r = dz_r W_e;   dW_e = sum over e's rows of dz_r x_t^T
#include <algorithm>

#include "common.h"
#include "grouped_common.h"
#include "grouped_mma.h"
#include "linear_common.h"

namespace moe {
namespace grp {

constexpr int TILE = 64, BK = 16, PITCH = TILE + 4;

// 64 x 64 outputs per workgroup, 4 x 4 per thread, operands through LDS as
// fp32, the reduction's elements outside the matrix as zeros.
template <typename E, int MODE, bool GLU>
__global__ __launch_bounds__(256) void simple_kernel(Prod p, int col_tiles, long tiles) {
  __shared__ float sr[BK][PITCH], sc[GLU ? 2 : 1][BK][PITCH];
  const E *R = static_cast<const E*>(p.r), *C = static_cast<const E*>(p.c);
  const int O = GLU ? p.W / 2 : p.W;
  const int M_dw = (p.W + TILE - 1) / TILE;
  for (long at = blockIdx.x; at < tiles; at += gridDim.x) {
    int e, lo, hi, m0;
    const int n0 = static_cast<int>(at % col_tiles) * TILE;
    if (MODE == DW) {
      const int rest = static_cast<int>(at / col_tiles);
      e = rest / M_dw;
      m0 = rest % M_dw * TILE;
      const Span s = span_of(p.g, e);
      lo = s.lo;
      hi = s.hi;
    } else {
      const RowTile t = row_tile(p.g, TILE, static_cast<int>(at / col_tiles));
      if (t.e < 0) return;
      e = t.e;
      lo = t.lo + t.tile * TILE;
      hi = min(t.hi, lo + TILE);
      m0 = 0;
    }
    const int N = MODE == FWD ? O : p.K;                        // output columns
    const int len = MODE == DW ? hi - lo : MODE == FWD ? p.K : p.W;  // reduction
    const E* we = C + static_cast<size_t>(e) * p.W * p.K;
    float acc[GLU ? 2 : 1][4][4] = {};
    const int tm = threadIdx.x / 16 * 4, tn = threadIdx.x % 16 * 4;
    for (int k0 = 0; k0 < len; k0 += BK) {
      __syncthreads();
      for (int i = threadIdx.x; i < TILE * BK; i += 256) {
        // along memory: k for reduction-contiguous operands, m or n otherwise
        const int kc = i % BK, mc = i / BK, ks = i / TILE, ms = i % TILE;
        if (MODE == DW) {
          const int r = lo + k0 + ks;
          const bool in = k0 + ks < len;
          sr[ks][ms] = in && m0 + ms < p.W ? load1(R + static_cast<size_t>(r) * p.W + m0 + ms) : 0.f;
          const int xr = in && p.token ? p.token[r] : r;
          sc[0][ks][ms] = in && n0 + ms < N ? load1(C + static_cast<size_t>(xr) * p.K + n0 + ms) : 0.f;
        } else {
          const int r = lo + mc;
          const bool in = r < hi && k0 + kc < len;
          const int xr = in && MODE == FWD && p.token ? p.token[r] : r;
          sr[kc][mc] = in ? load1(R + static_cast<size_t>(xr) * len + k0 + kc) : 0.f;
          if (MODE == FWD) {
            const bool on = n0 + mc < N && k0 + kc < len;
            const size_t w = static_cast<size_t>(n0 + mc) * p.K + k0 + kc;
            sc[0][kc][mc] = on ? load1(we + w) : 0.f;
            if constexpr (GLU) sc[1][kc][mc] = on ? load1(we + w + static_cast<size_t>(O) * p.K) : 0.f;
          } else {
            sc[0][ks][ms] = n0 + ms < N && k0 + ks < len
                                ? load1(we + static_cast<size_t>(k0 + ks) * p.K + n0 + ms) : 0.f;
          }
        }
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < BK; ++k)
#pragma unroll
        for (int h = 0; h < (GLU ? 2 : 1); ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[h][i][j] += sr[k][tm + i] * sc[h][k][tn + j];
    }
    if (n0 + tn >= N) continue;
    Epilogue out = p.e;
    if (MODE == DW) out.y = static_cast<E*>(p.e.y) + static_cast<size_t>(e) * p.W * p.K;
    for (int i = 0; i < 4; ++i) {
      const int m = MODE == DW ? m0 + tm + i : lo + tm + i;
      if (m >= (MODE == DW ? p.W : hi)) continue;
      finish<E, GLU, 4>(out, m, n0 + tn, N, acc[0][i], acc[GLU ? 1 : 0][i]);
    }
  }
}

// dz of the rows that the experts have, rounded to the element type: 16 bytes of
// dy's columns per thread.
template <typename D>
__global__ __launch_bounds__(256) void act_grad_kernel(const typename D::elem* __restrict__ dy,
                                                       const typename D::elem* __restrict__ z,
                                                       Groups g, int O, int act,
                                                       typename D::elem* __restrict__ dz) {
  constexpr int V = D::V;
  const unsigned cols = O / V;
  const size_t M = max(0, min(g.offsets[g.N], g.R));
  const size_t n = M * cols, step = gridDim.x * static_cast<size_t>(256);
  const bool glu = act == MOE_ACT_SWIGLU;
  for (size_t i = blockIdx.x * static_cast<size_t>(256) + threadIdx.x; i < n; i += step) {
    const size_t t = i / cols, o = (i - t * cols) * V;
    const size_t zr = t * (glu ? 2 * static_cast<size_t>(O) : O) + o;
    float d[V], up[V];
    act_grad<typename D::elem, V>(dy + i * V, z + zr, O, act, d, up);
    store_v<V>(dz + zr, d);
    if (glu) store_v<V>(dz + zr + O, up);
  }
}

// --------------------------------------------------------------------- host
inline size_t elem_size(int dtype) { return dtype == MOE_BF16 ? 2 : 4; }
inline int width(int O, int act) { return act == MOE_ACT_SWIGLU ? 2 * O : O; }

inline int check(int R, int N, int K, int O, int act, int dtype) {
  if (R < 0 || R > MOE_GROUPED_MAX_ROWS || N < 1 || N > 1024 || K < 1 ||
      K > MOE_LINEAR_MAX_DIM || O < 1 || O > MOE_LINEAR_MAX_DIM || act < MOE_ACT_NONE ||
      act > MOE_ACT_SWIGLU)
    return MOE_EINVAL;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EUNSUP;
  const int step = dtype == MOE_BF16 ? 8 : 4;
  return K % step != 0 || O % step != 0 ? MOE_EUNSUP : MOE_OK;
}

// x is [T,K] behind row_token, else it holds the rows themselves
inline int check_tokens(const int32_t* row_token, int T, int R, int K, int dtype) {
  if (T < 0 || T > MOE_GROUPED_MAX_ROWS) return MOE_EINVAL;
  if (!row_token) return T == R ? MOE_OK : MOE_EINVAL;
  if (R > 0 && T == 0) return MOE_EINVAL;
  return static_cast<size_t>(T) * K * elem_size(dtype) > (size_t(1) << 31) ? MOE_EUNSUP : MOE_OK;
}

template <typename E, int MODE, bool GLU>
void launch(const Prod& p, hipStream_t s) {
  const int N = MODE == FWD ? (GLU ? p.W / 2 : p.W) : p.K, cols = (N + TILE - 1) / TILE;
  const long tiles = cols * (MODE == DW ? static_cast<long>(p.g.N) * ((p.W + TILE - 1) / TILE)
                                        : max_row_tiles(p.g.R, p.g.N, TILE));
  hipLaunchKernelGGL((simple_kernel<E, MODE, GLU>), dim3(std::min<long>(tiles, 1 << 20)), dim3(256), 0,
                     s, p, cols, tiles);
}

template <int MODE, int BM, int BN, int WGS, bool GLU, bool GATHER>
int launch_mma(const Prod& p, hipStream_t s) {
  constexpr int lds = (SA * BM + SB * BN) * SLICE * 2, NC = GLU ? BN / 2 : BN;
  const auto fn = grouped_mma_kernel<MODE, BM, BN, WGS, GLU, GATHER>;
  static std::atomic<bool> done[64];
  if (!allow_lds(reinterpret_cast<const void*>(fn), lds, done)) return MOE_EHIP;
  const int N = MODE == FWD ? (GLU ? p.W / 2 : p.W) : p.K;
  const long rows = MODE == DW ? static_cast<long>(p.g.N) * ((p.W + BM - 1) / BM)
                               : max_row_tiles(p.g.R, p.g.N, BM);
  const long tiles = rows * ((N + NC - 1) / NC);
  if (tiles > (1 << 23)) return MOE_EUNSUP;  // the outputs alone would not fit the card
  // DW: workgroups that stay; a short list may fall unevenly on the XCDs
  const long wgs = MODE == DW ? std::min<long>(WGS * cu_count(), 2 * tiles) : tiles;
  hipLaunchKernelGGL(fn, dim3(static_cast<unsigned>((wgs + 7) / 8 * 8)), dim3(lin::W * MOE_WAVE), lds,
                     s, p);
  return MOE_OK;
}

template <int MODE, bool GLU>
int launch_bf16(const Prod& p, hipStream_t s) {
  // rows of an expert: a 256-row tile is half empty for 128
  const bool large = p.g.R / p.g.N >= 192;
  if (MODE != DX && p.token)
    return large ? launch_mma<MODE, 256, 256, 1, GLU, MODE != DX>(p, s)
                 : launch_mma<MODE, 128, 128, 2, GLU, MODE != DX>(p, s);
  return large ? launch_mma<MODE, 256, 256, 1, GLU, false>(p, s)
               : launch_mma<MODE, 128, 128, 2, GLU, false>(p, s);
}

// Product of any type
template <typename E, int MODE, bool GLU>
int product(const Prod& p, hipStream_t s) {
  if constexpr (sizeof(E) == 2) return launch_bf16<MODE, GLU>(p, s);
  launch<E, MODE, GLU>(p, s);
  return MOE_OK;
}

inline size_t dz_bytes(int R, int O, int act, int dtype) {
  return act == MOE_ACT_NONE ? 0 : static_cast<size_t>(R) * width(O, act) * elem_size(dtype);
}

template <typename D>
int backward(const void* dy, const void* x, const int32_t* row_token, const Groups& g,
             const void* w, const void* z, int T, int K, int O, int act, void* dx, void* dw, void* ws,
             hipStream_t s) {
  typedef typename D::elem E;
  const int W = width(O, act);
  if (g.R == 0) {  // sums over no rows
    if (!dw) return MOE_OK;
    const size_t n = static_cast<size_t>(g.N) * W * K;
    hipLaunchKernelGGL(zero_kernel<E>, grid_of(n), dim3(256), 0, s, static_cast<E*>(dw), n);
    return launch_status();
  }
  const void* dz = dy;
  if (act != MOE_ACT_NONE) {
    dz = ws;
    const size_t chunks = static_cast<size_t>(g.R) * (O / D::V);
    hipLaunchKernelGGL(act_grad_kernel<D>, grid_of(chunks), dim3(256), 0, s,
                       static_cast<const E*>(dy), static_cast<const E*>(z), g, O, act,
                       static_cast<E*>(ws));
  }
  Prod p{dz, w, nullptr, 0, g, W, K, Epilogue{}};
  p.e.y = dx;
  int rc = dx ? product<E, DX, false>(p, s) : MOE_OK;
  p.c = x;
  p.token = row_token;
  p.x_rows = T;
  p.e.y = dw;
  if (dw && rc == MOE_OK) rc = product<E, DW, false>(p, s);
  return rc == MOE_OK ? launch_status() : rc;
}

}  // namespace grp
}  // namespace moe

using namespace moe;
using namespace moe::grp;

extern "C" size_t moe_grouped_linear_workspace_size(int R, int N, int K, int O, int act, int dtype) {
  return check(R, N, K, O, act, dtype) == MOE_OK ? 256 : 0;
}

extern "C" int moe_grouped_linear(const void* x, const int32_t* row_token,
                                  const int32_t* expert_offsets, const void* w, int T, int R, int N,
                                  int K, int O, int act, int dtype, void* z, void* y,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check(R, N, K, O, act, dtype);
  if (rc == MOE_OK) rc = check_tokens(row_token, T, R, K, dtype);
  if (rc != MOE_OK || R == 0) return rc;
  if (!x || !expert_offsets || !w || !y || !workspace ||
      workspace_bytes < moe_grouped_linear_workspace_size(R, N, K, O, act, dtype))
    return MOE_EINVAL;
  for (const void* q : {x, w, static_cast<const void*>(z), static_cast<const void*>(y),
                        static_cast<const void*>(workspace)})
    if (!aligned16(q)) return MOE_EINVAL;
  hipStream_t s = as_stream(stream);
  const Prod p{x, w, row_token, static_cast<size_t>(T), Groups{expert_offsets, N, R}, width(O, act), K,
               Epilogue{nullptr, nullptr, z, y, act}};
  const bool glu = act == MOE_ACT_SWIGLU;
  rc = dtype == MOE_BF16
           ? (glu ? product<uint16_t, FWD, true>(p, s) : product<uint16_t, FWD, false>(p, s))
           : (glu ? product<float, FWD, true>(p, s) : product<float, FWD, false>(p, s));
  return rc == MOE_OK ? launch_status() : rc;
}

extern "C" size_t moe_grouped_linear_backward_workspace_size(int R, int N, int K, int O, int act,
                                                             int dtype) {
  if (check(R, N, K, O, act, dtype) != MOE_OK) return 0;
  return dz_bytes(R, O, act, dtype) + 256;
}

extern "C" int moe_grouped_linear_backward(const void* dy, const void* x, const int32_t* row_token,
                                           const int32_t* expert_offsets, const void* w,
                                           const void* z, int T, int R, int N, int K, int O,
                                           int act, int dtype, void* dx, void* dw, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  int rc = check(R, N, K, O, act, dtype);
  if (rc == MOE_OK && (x || dw)) rc = check_tokens(row_token, T, R, K, dtype);
  if (rc != MOE_OK) return rc;
  if (R > 0 && ((!dx && !dw) || !dy || !expert_offsets || (act != MOE_ACT_NONE && !z) ||
                (dx && !w) || (dw && !x) || !workspace ||
                workspace_bytes < moe_grouped_linear_backward_workspace_size(R, N, K, O, act, dtype)))
    return MOE_EINVAL;
  for (const void* q : {dy, x, w, z, static_cast<const void*>(dx), static_cast<const void*>(dw),
                        static_cast<const void*>(workspace)})
    if (!aligned16(q)) return MOE_EINVAL;
  const Groups g{expert_offsets, N, R};
  hipStream_t s = as_stream(stream);
  return dtype == MOE_BF16
             ? backward<Bf16>(dy, x, row_token, g, w, z, T, K, O, act, dx, dw, workspace, s)
             : backward<F32>(dy, x, row_token, g, w, z, T, K, O, act, dx, dw, workspace, s);
}
