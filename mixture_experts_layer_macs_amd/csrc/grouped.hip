// moe_grouped_linear and moe_grouped_linear_backward: the routed experts'
// products over ragged groups of rows, and their gradients.
//
//   z_r = W_e x_t,  y_r = act(z_r);   dz = dy act'(z)
//   dx_r = dz_r W_e;   dW_e = sum over e's rows of dz_r x_t^T
#include <algorithm>

#include "common.h"
#include "grouped_common.h"
#include "grouped_f32.h"
#include "grouped_mma.h"
#include "grouped_plan.h"
#include "grouped_stream.h"
#include "linear_common.h"

namespace moe {
namespace grp {

// dz of the rows that the experts have, rounded to the element type: 16 bytes of
// dy's columns per thread; bound by HBM (65536 x 768 swiglu: 89 us, 5.6 TB/s).
template <typename D>
__device__ __forceinline__ void act_grad_rows(const typename D::elem* dy, const typename D::elem* z,
                                              const Groups& g, int O, int act, typename D::elem* dz,
                                              unsigned block, unsigned blocks) {
  constexpr int V = D::V;
  const unsigned cols = O / V;
  const size_t M = max(0, min(g.offsets[g.N], g.R));
  const size_t n = M * cols, step = blocks * static_cast<size_t>(256);
  const bool glu = act == MOE_ACT_SWIGLU;
  for (size_t i = block * static_cast<size_t>(256) + threadIdx.x; i < n; i += step) {
    const size_t t = i / cols, o = (i - t * cols) * V;
    const size_t zr = t * (glu ? 2 * static_cast<size_t>(O) : O) + o;
    float d[V], up[V];
    act_grad<typename D::elem, V>(dy + i * V, z + zr, O, act, d, up);
    store_v<V>(dz + zr, d);
    if (glu) store_v<V>(dz + zr + O, up);
  }
}

// The rows of x in the experts' order, for the reduction over them: a gather
// inside the product, along the axis that it reduces, cost it 20 to 37 % (8192
// tokens, 128 experts, 1536 x 2048: 743 us for 543), this copy 75 us beside the
// activation gradient.
struct Gathered {
  const uint16_t* x;
  const int32_t* token;
  uint16_t* rows;
  int K;
};
__device__ __forceinline__ void gather_rows(const Gathered& a, const Groups& g, unsigned block,
                                            unsigned blocks) {
  const unsigned cols = a.K / 8;
  const size_t M = max(0, min(g.offsets[g.N], g.R));
  const size_t n = M * cols, step = blocks * static_cast<size_t>(256);
  for (size_t i = block * static_cast<size_t>(256) + threadIdx.x; i < n; i += step) {
    const size_t r = i / cols, c = i - r * cols;
    reinterpret_cast<u32x4*>(a.rows)[i] =
        *reinterpret_cast<const u32x4*>(a.x + static_cast<size_t>(a.token[r]) * a.K + c * 8);
  }
}

// What the products read: the plan of the streaming ones, by the first workgroup,
// dz, by the next `own`, and the gathered rows, by the others.
template <typename D>
__global__ __launch_bounds__(256) void prepare_kernel(const typename D::elem* dy,
                                                      const typename D::elem* z, Groups g, int O,
                                                      int act, typename D::elem* dz, unsigned own,
                                                      Gathered a, Plan* plan) {
  const unsigned block = blockIdx.x - 1;
  if (blockIdx.x == 0) {
    if (plan) make_plan(g, plan);
  } else if (block < own) {
    act_grad_rows<D>(dy, z, g, O, act, dz, block, own);
  } else {
    gather_rows(a, g, block - own, gridDim.x - 1 - own);
  }
}

// The parts' sums, in their order, to dw.
__global__ __launch_bounds__(256) void join_weights_kernel(Prod p, size_t quads) {
  const size_t step = gridDim.x * static_cast<size_t>(256);
  for (size_t i = blockIdx.x * static_cast<size_t>(256) + threadIdx.x; i < quads; i += step) {
    float v[4] = {};
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
      float f[4];
      load4(p.part + (s * quads + i) * 4, f);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += f[j];
    }
    store4(static_cast<uint16_t*>(p.e.y) + i * 4, v);
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

template <int MODE, int BM, int BN, int SL, int RA, int WGS, bool GLU, bool GATHER>
int launch_mma(const Prod& p, hipStream_t s) {
  constexpr int lds = (RA * BM + SB * BN) * SL * 2, NC = GLU ? BN / 2 : BN;
  const auto fn = grouped_mma_kernel<MODE, BM, BN, SL, RA, WGS, GLU, GATHER>;
  const int N = MODE == FWD ? (GLU ? p.W / 2 : p.W) : p.K;
  const long rows = MODE == DW ? static_cast<long>(p.g.N) * ((p.W + BM - 1) / BM)
                               : max_row_tiles(p.g.R, p.g.N, BM);
  const long tiles = rows * ((N + NC - 1) / NC) * (MODE == DW && GLU ? p.splits : 1);
  if (tiles > MOE_GROUPED_MAX_TILES) return MOE_EUNSUP;  // a grid holds fewer than 2^32 threads
  static std::atomic<bool> done[64];
  if (!allow_lds(reinterpret_cast<const void*>(fn), lds, done)) return MOE_EHIP;
  hipLaunchKernelGGL(fn, dim3(static_cast<unsigned>((tiles + 7) / 8 * 8)), dim3(lin::W * MOE_WAVE), lds,
                     s, p);
  return MOE_OK;
}

template <int MODE>
int launch_stream(const Prod& p, Plan* plan, hipStream_t s) {
  const auto fn = grouped_stream_mma_kernel<MODE>;
  static std::atomic<bool> done[64];
  if (!allow_lds(reinterpret_cast<const void*>(fn), ST_LDS, done)) return MOE_EHIP;
  hipLaunchKernelGGL(fn, dim3((cu_count() + 7) / 8 * 8), dim3(lin::W * MOE_WAVE),
                     ST_LDS, s, p, plan);
  return MOE_OK;
}

inline bool streams(int mode, const Prod& p) {
  return tile_choice(mode, p.g.R, p.g.N, p.W, p.K, cu_count()) == STREAM;
}

template <bool GLU, bool GATHER>
int launch_skinny(const Prod& p, hipStream_t s) {
  constexpr int NC = GLU ? 8 : 16;
  const int O = GLU ? p.W / 2 : p.W;
  const long tiles = max_row_tiles(p.g.R, p.g.N, 16) * ((O + NC - 1) / NC);
  hipLaunchKernelGGL((grouped_skinny_kernel<GLU, GATHER>), dim3(static_cast<unsigned>((tiles + 7) / 8 * 8)),
                     dim3(SK_WAVES * MOE_WAVE), 0, s, p);
  return MOE_OK;
}

// plan: of the streaming products
template <int MODE, bool GLU, bool GATHER>
int launch_tile(const Prod& p, Plan* plan, hipStream_t s) {
  switch (tile_choice(MODE, p.g.R, p.g.N, p.W, p.K, cu_count())) {
    case STREAM:
      if constexpr (MODE != FWD) return launch_stream<MODE>(p, plan, s);
    case SKINNY:
      if constexpr (MODE == FWD) return launch_skinny<GLU, GATHER>(p, s);
    case TILE_256: return launch_mma<MODE, 256, 256, 64, 2, 1, GLU, GATHER>(p, s);
    case TILE_128x256:
      if constexpr (MODE == DX) return launch_mma<MODE, 128, 256, 32, 3, 2, GLU, GATHER>(p, s);
    default:
      if constexpr (MODE == DW)
        if (p.splits > 1) {
          const int rc = launch_mma<DW, 128, 128, 64, 2, 2, true, false>(p, s);
          const size_t quads = static_cast<size_t>(p.g.N) * p.W * p.K / 4;
          if (rc == MOE_OK)
            hipLaunchKernelGGL(join_weights_kernel, grid_of(quads), dim3(256), 0, s, p, quads);
          return rc;
        }
      return launch_mma<MODE, 128, 128, 64, 2, 2, GLU, GATHER>(p, s);
  }
}

template <int MODE, bool GLU>
int launch_bf16(const Prod& p, Plan* plan, hipStream_t s) {
  if constexpr (MODE == FWD)
    if (p.token) return launch_tile<MODE, GLU, true>(p, plan, s);
  return launch_tile<MODE, GLU, false>(p, plan, s);
}

template <int MODE>
long f32_tiles(const Prod& p, bool glu, int edge) {
  const int nc = glu && edge > 32 ? edge / 2 : edge, N = MODE == FWD ? (glu ? p.W / 2 : p.W) : p.K;
  const long rows = MODE == DW ? static_cast<long>(p.g.N) * ((p.W + edge - 1) / edge)
                               : max_row_tiles(p.g.R, p.g.N, edge);
  return (rows * ((N + nc - 1) / nc) + 7) / 8 * 8;
}

template <int MODE, bool GLU, bool GATHER, int EDGE>
int launch_f32_tile(const Prod& p, hipStream_t s) {
  const long tiles = f32_tiles<MODE>(p, GLU, EDGE);
  if (tiles > INT32_MAX) return MOE_EUNSUP;  // the outputs alone would not fit the card
  hipLaunchKernelGGL((grouped_f32_kernel<MODE, GLU, GATHER, EDGE>),
                     dim3(static_cast<unsigned>(std::min<long>(tiles, 1 << 20))), dim3(256), 0, s, p,
                     static_cast<int>(tiles));
  return MOE_OK;
}

template <int MODE, bool GLU, bool GATHER>
int launch_f32_edge(const Prod& p, hipStream_t s) {
  const int edge = tile_choice_f32(MODE, p.g.R, p.g.N, p.W, p.K, cu_count());
  return edge == 32   ? launch_f32_tile<MODE, GLU, GATHER, 32>(p, s)
         : edge == 64 ? launch_f32_tile<MODE, GLU, GATHER, 64>(p, s)
                      : launch_f32_tile<MODE, GLU, GATHER, 128>(p, s);
}

template <int MODE, bool GLU>
int launch_f32(const Prod& p, hipStream_t s) {
  if constexpr (MODE != DX)
    if (p.token) return launch_f32_edge<MODE, GLU, true>(p, s);
  return launch_f32_edge<MODE, GLU, false>(p, s);
}

// Product of any type
template <typename E, int MODE, bool GLU>
int product(const Prod& p, Plan* plan, hipStream_t s) {
  if constexpr (sizeof(E) == 2) return launch_bf16<MODE, GLU>(p, plan, s);
  else return launch_f32<MODE, GLU>(p, s);
}

// dx and dw (either may be absent: null y)
template <typename E>
int products(const Prod& x, const Prod& w, Plan* plan, hipStream_t s) {
  if (sizeof(E) == 4 && x.e.y && w.e.y) {
    const int cus = cu_count();
    const long dw0 = f32_tiles<DX>(x, false, 32), all = dw0 + f32_tiles<DW>(w, false, 32);
    if (tile_choice_f32(DX, x.g.R, x.g.N, x.W, x.K, cus) == 32 &&
        tile_choice_f32(DW, x.g.R, x.g.N, x.W, x.K, cus) == 32 && all <= (1 << 20)) {
      const dim3 grid(static_cast<unsigned>(all)), block(256);
      if (w.token)
        hipLaunchKernelGGL((grouped_f32_pair_kernel<true>), grid, block, 0, s, x, w, static_cast<int>(dw0));
      else
        hipLaunchKernelGGL((grouped_f32_pair_kernel<false>), grid, block, 0, s, x, w, static_cast<int>(dw0));
      return MOE_OK;
    }
  }
  int rc = x.e.y ? product<E, DX, false>(x, plan, s) : MOE_OK;
  if (w.e.y && rc == MOE_OK) rc = product<E, DW, false>(w, plan, s);
  return rc;
}

// Parts of the weight gradient's reduction.
inline int splits_of(int R, int N, int W, int K, int dtype) {
  const int cus = cu_count();
  return dtype == MOE_BF16 && R > 0 && tile_choice(DW, R, N, W, K, cus) == TILE_128
             ? split_choice(R, N, W, K, cus) : 1;
}

// The backward pass's workspace: dz, then (bf16) the rows of x, the plan and the
// parts of dw.
struct BackSpace {
  size_t rows, plan, part, bytes;
  int splits;
};
inline BackSpace back_space(int R, int N, int K, int O, int act, int dtype) {
  const size_t el = elem_size(dtype);
  const size_t dz = act == MOE_ACT_NONE ? 0 : (R * (width(O, act) * el) + 255) / 256 * 256;
  const size_t rows = dtype == MOE_BF16 ? (static_cast<size_t>(R) * K * el + 255) / 256 * 256 : 0;
  const size_t part = dz + rows + (sizeof(Plan) + 255) / 256 * 256;
  const int splits = splits_of(R, N, width(O, act), K, dtype);
  return {dz, dz + rows, part,
          part + (splits > 1 ? static_cast<size_t>(splits) * N * width(O, act) * K * 4 : 0), splits};
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
  char* space = static_cast<char*>(ws);
  const void* dz = act == MOE_ACT_NONE ? dy : ws;
  const BackSpace b = back_space(g.R, g.N, K, O, act, sizeof(E) == 2 ? MOE_BF16 : MOE_F32);
  Gathered a{};
  if (sizeof(E) == 2 && row_token && dw) {
    a = Gathered{static_cast<const uint16_t*>(x), row_token, reinterpret_cast<uint16_t*>(space + b.rows), K};
    x = a.rows;
    row_token = nullptr;
  }
  Prod px{dz, w, nullptr, 0, g, W, K, Epilogue{}};
  Prod pw{dz, x, row_token, static_cast<size_t>(T), g, W, K, Epilogue{}};
  px.e.y = dx;
  pw.e.y = dw;
  pw.splits = b.splits;
  pw.part = reinterpret_cast<float*>(space + b.part);
  Plan* plan = nullptr;
  if (sizeof(E) == 2 && ((dx && streams(DX, px)) || (dw && streams(DW, pw))))
    plan = reinterpret_cast<Plan*>(space + b.plan);
  const unsigned own = act == MOE_ACT_NONE ? 0 : grid_of(static_cast<size_t>(g.R) * (O / D::V)).x;
  const unsigned copy = a.rows ? grid_of(static_cast<size_t>(g.R) * (K / 8)).x : 0;
  if (own + copy || plan)
    hipLaunchKernelGGL(prepare_kernel<D>, dim3(1 + own + copy), dim3(256), 0, s,
                       static_cast<const E*>(dy), static_cast<const E*>(z), g, O, act,
                       static_cast<E*>(ws), own, a, plan);
  const int rc = products<E>(px, pw, plan, s);
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
           ? (glu ? product<uint16_t, FWD, true>(p, nullptr, s) : product<uint16_t, FWD, false>(p, nullptr, s))
           : (glu ? product<float, FWD, true>(p, nullptr, s) : product<float, FWD, false>(p, nullptr, s));
  return rc == MOE_OK ? launch_status() : rc;
}

extern "C" size_t moe_grouped_linear_backward_workspace_size(int R, int N, int K, int O, int act,
                                                             int dtype) {
  if (check(R, N, K, O, act, dtype) != MOE_OK) return 0;
  return back_space(R, N, K, O, act, dtype).bytes;
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
