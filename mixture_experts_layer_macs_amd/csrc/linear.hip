// moe_linear and moe_linear_backward: the matrix product of the dense parts
// beside the routed experts, with bias, activation and residual in its
// epilogue, and its gradients.
//
//   z = x W^T + b,   y = act(z) + residual
//   dz = dy act'(z);   dx = dz W,   dW = dz^T x,   db = sum_t dz
//
// act "swiglu" takes W [2O,K], gate rows first: y = silu(z[:, :O]) z[:, O:].
#include <algorithm>
#include <atomic>

#include "common.h"
#include "linear_common.h"
#include "linear_f32.h"
#include "linear_mma.h"
#include "linear_plan.h"
#include "linear_skinny.h"

namespace moe {
namespace lin {

// ------------------------------------------------------------ bf16 product
// The LDS limit is a per-device function attribute: set once per device.
inline bool allow_lds(const void* fn, int bytes, std::atomic<bool>* done) {
  const int dev = current_device();
  if (dev >= 0 && done[dev].load(std::memory_order_acquire)) return true;
  if (hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, bytes) != hipSuccess)
    return false;
  if (dev >= 0) done[dev].store(true, std::memory_order_release);
  return true;
}

inline int grid_of(const Mma& a) { return (a.tm * a.tn * a.splits + 7) / 8 * 8; }

template <bool RS, bool CS, int BM, int BN, int WGS, bool GLU, bool PART>
int launch_mma(const Mma& a, hipStream_t s) {
  constexpr int lds = (SA * BM + SB * BN) * SLICE * 2;
  const auto fn = mma_kernel<RS, CS, BM, BN, WGS, GLU, PART>;
  static std::atomic<bool> done[64];
  if (!allow_lds(reinterpret_cast<const void*>(fn), lds, done)) return MOE_EHIP;
  hipLaunchKernelGGL(fn, dim3(grid_of(a)), dim3(W * MOE_WAVE), lds, s, a);
  return MOE_OK;
}

// Sums the splits' partial products in their order and finishes the output.
// GLU: the parts hold gate and up columns, 2 N of them.
template <typename E, bool GLU>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ part, int splits,
                                                   int M, int N, Epilogue e) {
  const size_t i = (blockIdx.x * static_cast<size_t>(256) + threadIdx.x) * 4;
  if (i >= static_cast<size_t>(M) * N) return;
  const int m = static_cast<int>(i / N), n = static_cast<int>(i % N);
  const size_t W = GLU ? 2 * static_cast<size_t>(N) : N;
  float g[4] = {}, u[4] = {};
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float* p = part + (static_cast<size_t>(s) * M + m) * W + n;
    float f[4];
    load4(p, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) g[j] += f[j];
    if constexpr (GLU) {
      load4(p + N, f);
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] += f[j];
    }
  }
  finish<E, GLU, 4>(e, m, n, N, g, u);
}

// The plan's tiles and splits of a product of W output columns (GLU: gate and
// up) in `a`; part: room for the partial sums.
inline void cut(Mma& a, const Plan& p, int W, float* part) {
  a.per_split = ((a.K + p.splits - 1) / p.splits + 63) / 64 * 64;
  a.splits = (a.K + a.per_split - 1) / a.per_split;
  a.tm = (a.M + TILES[p.tile].m - 1) / TILES[p.tile].m;
  a.tn = (W + TILES[p.tile].n - 1) / TILES[p.tile].n;
  a.part = part;
}

template <bool RS, bool CS, bool GLU, bool PART>
int launch_tile(const Mma& a, int tile, hipStream_t s) {
  switch (tile) {
    case 0: return launch_mma<RS, CS, 256, 256, 1, GLU, PART>(a, s);
    case 1: return launch_mma<RS, CS, 256, 192, 1, GLU, PART>(a, s);
    case 2: return launch_mma<RS, CS, 192, 256, 1, GLU, PART>(a, s);
    default: return launch_mma<RS, CS, 128, 128, 2, GLU, PART>(a, s);
  }
}

template <typename E, bool GLU>
void launch_join(const float* part, int splits, int M, int N, const Epilogue& e, hipStream_t s) {
  const size_t quads = static_cast<size_t>(M) * N / 4;
  hipLaunchKernelGGL((join_kernel<E, GLU>), dim3((quads + 255) / 256), dim3(256), 0, s, part, splits,
                     M, N, e);
}

template <bool RS, bool CS, bool GLU>
int product(Mma a, const Plan& p, float* part, hipStream_t s) {
  const int N = a.N, W = GLU ? 2 * N : N;
  cut(a, p, W, part);
  if (a.splits == 1) return launch_tile<RS, CS, GLU, false>(a, p.tile, s);
  a.N = W;
  const int rc = launch_tile<RS, CS, false, true>(a, p.tile, s);
  if (rc == MOE_OK) launch_join<uint16_t, GLU>(part, a.splits, a.M, N, a.e, s);
  return rc;
}

// ------------------------------------------------------------ fp32 product
template <bool RS, bool CS, bool GLU>
int product_f32(F32Prod a, const Plan& p, float* part, hipStream_t s) {
  if (p.tile == 32) {
    hipLaunchKernelGGL((f32_small_kernel<RS, CS, GLU>), dim3((a.N + 31) / 32, (a.M + 31) / 32),
                       dim3(256), 0, s, a);
    return MOE_OK;
  }
  a.per_split = ((a.K + p.splits - 1) / p.splits + 31) / 32 * 32;
  const int splits = (a.K + a.per_split - 1) / a.per_split, N = a.N;
  a.part = part;
  if (splits == 1) {
    const int nc = GLU ? p.tile / 2 : p.tile;
    const dim3 grid((N + nc - 1) / nc, (a.M + p.tile - 1) / p.tile);
    if (p.tile == 64)
      hipLaunchKernelGGL((f32_large_kernel<RS, CS, 1, GLU, false>), grid, dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((f32_large_kernel<RS, CS, 2, GLU, false>), grid, dim3(256), 0, s, a);
    return MOE_OK;
  }
  if (GLU) a.N *= 2;
  const dim3 grid((a.N + p.tile - 1) / p.tile, (a.M + p.tile - 1) / p.tile, splits);
  if (p.tile == 64)
    hipLaunchKernelGGL((f32_large_kernel<RS, CS, 1, false, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((f32_large_kernel<RS, CS, 2, false, true>), grid, dim3(256), 0, s, a);
  launch_join<float, GLU>(part, splits, a.M, N, a.e, s);
  return MOE_OK;
}

// ----------------------------------------------------------- few tokens
template <bool GLU>
int launch_skinny(Skinny p, int rf, hipStream_t s) {
  p.panels = GLU ? (p.O + 7) / 8 : (p.O + 15) / 16;
  p.parts = (p.T + rf * 16 - 1) / (rf * 16);
  const dim3 grid((p.panels * p.parts + 7) / 8 * 8), block(SK_WAVES * MOE_WAVE);
  if (rf == 1) hipLaunchKernelGGL((skinny_kernel<1, GLU>), grid, block, 0, s, p);
  else if (rf == 2) hipLaunchKernelGGL((skinny_kernel<2, GLU>), grid, block, 0, s, p);
  else if (rf == 4) hipLaunchKernelGGL((skinny_kernel<4, GLU>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((skinny_kernel<8, GLU>), grid, block, 0, s, p);
  return MOE_OK;
}

// ------------------------------------------------ activation gradient, bias
// dz of V consecutive columns from dy and z, in fp32.  GLU: g ends as the gate
// half and up as the up half.
template <typename E, int V>
__device__ __forceinline__ void act_grad(const E* dy, const E* z, int O, int act, float* g,
                                         float* up) {
  load_v<V>(dy, g);
  if (act == MOE_ACT_NONE) return;
  float a[V];
  load_v<V>(z, a);
  if (act == MOE_ACT_SWIGLU) {
    load_v<V>(z + O, up);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float sg = sigmoid(a[i]), d = g[i] * silu(a[i], sg);
      g[i] *= up[i] * silu_slope(a[i], sg);
      up[i] = d;
    }
  } else if (act == MOE_ACT_RELU) {  // a closed unit passes nothing, whatever dy is
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = a[i] <= 0.f ? 0.f : g[i];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] *= act_slope<E>(act, a[i]);
  }
}

// dz rounded to the element type, the operand of both products: 16 bytes of
// dy's columns per thread.  Bound by HBM: dy and z read, dz written once (8192 x
// 768 swiglu: 13 us, 63 MB, 4.8 TB/s).  bf16 is what the matrix instructions
// multiply: x, w and the results have that type, and dz kept as two bf16 terms
// would double the products, 110 of the 128 us.  It is the only rounding between
// dy and the sums; dx and dw end 2.35e-3 off in the 2-norm, where rounding the
// results alone gives 1.66e-3.
template <typename D>
__global__ __launch_bounds__(256) void act_grad_kernel(const typename D::elem* __restrict__ dy,
                                                       const typename D::elem* __restrict__ z,
                                                       int T, int O, int act,
                                                       typename D::elem* __restrict__ dz) {
  constexpr int V = D::V;
  const unsigned cols = O / V;
  const size_t n = static_cast<size_t>(T) * cols, step = gridDim.x * static_cast<size_t>(256);
  const bool glu = act == MOE_ACT_SWIGLU;
  for (size_t i = blockIdx.x * static_cast<size_t>(256) + threadIdx.x; i < n; i += step) {
    const unsigned t = i / cols, o = (i - static_cast<size_t>(t) * cols) * V;
    const size_t zr = static_cast<size_t>(t) * (glu ? 2 * O : O) + o;
    float g[V], up[V];
    act_grad<typename D::elem, V>(dy + i * V, z + zr, O, act, g, up);
    store_v<V>(dz + zr, g);
    if (glu) store_v<V>(dz + zr + O, up);
  }
}

// The same with, per block of token rows, the fp32 column sums of the unrounded
// dz: a thread owns 16 bytes of dy's columns in every eighth row of the block.
constexpr int COLT = 32;  // threads along the columns; ROWT along the rows

template <typename D>
__global__ __launch_bounds__(COLT * ROWT) void act_grad_sum_kernel(
    const typename D::elem* __restrict__ dy, const typename D::elem* __restrict__ z, int T, int O,
    int act, int rows, typename D::elem* __restrict__ dz, float* __restrict__ part) {
  constexpr int V = D::V;
  __shared__ float red[ROWT][COLT * V];
  const int cx = threadIdx.x % COLT, ry = threadIdx.x / COLT;
  const int o = (blockIdx.x * COLT + cx) * V;
  const bool live = o < O, glu = act == MOE_ACT_SWIGLU;
  const int W = glu ? 2 * O : O;
  float s0[V] = {}, s1[V] = {};
  const int t0 = blockIdx.y * rows, t1 = min(T, t0 + rows);
  for (int t = live ? t0 + ry : t1; t < t1; t += ROWT) {
    const size_t zr = static_cast<size_t>(t) * W + o;
    float g[V], up[V];
    act_grad<typename D::elem, V>(dy + static_cast<size_t>(t) * O + o, z + zr, O, act, g, up);
    if (act != MOE_ACT_NONE) store_v<V>(dz + zr, g);
    if (glu) store_v<V>(dz + zr + O, up);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s0[i] += g[i];
      if (glu) s1[i] += up[i];
    }
  }
  for (int half = 0; half < (glu ? 2 : 1); ++half) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) red[ry][cx * V + i] = half ? s1[i] : s0[i];
    __syncthreads();
    for (int c = threadIdx.x; c < COLT * V; c += COLT * ROWT) {
      const int col = blockIdx.x * COLT * V + c;
      if (col >= O) continue;
      float v = 0.f;
#pragma unroll
      for (int r = 0; r < ROWT; ++r) v += red[r][c];
      part[static_cast<size_t>(blockIdx.y) * W + half * O + col] = v;
    }
  }
}

template <typename E>
__global__ __launch_bounds__(256) void bias_sum_kernel(BiasSum b) {
  __shared__ float red[256];
  bias_sum<E>(b, blockIdx.x, red);
}

template <typename E>
__global__ void zero_kernel(E* p, size_t n) {
  const size_t step = gridDim.x * static_cast<size_t>(256);
  for (size_t i = blockIdx.x * static_cast<size_t>(256) + threadIdx.x; i < n; i += step)
    store1(p + i, 0.f);
}

// --------------------------------------------------------------------- host
// Workgroups of 256 threads for n items; kernels loop over what is left beyond
// 2^22 of them (a grid holds fewer than 2^32 threads).
inline dim3 grid_of(size_t n) {
  return dim3(static_cast<unsigned>(std::min<size_t>((n + 255) / 256, size_t(1) << 22)));
}
inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

inline int check(int T, int K, int O, int act, int dtype) {
  if (T < 0 || T > (1 << 20) || K < 1 || K > MOE_LINEAR_MAX_DIM || O < 1 ||
      O > MOE_LINEAR_MAX_DIM || act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU)
    return MOE_EINVAL;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EUNSUP;
  const int step = dtype == MOE_BF16 ? 8 : 4;
  if (K % step != 0 || O % step != 0) return MOE_EUNSUP;
  return MOE_OK;
}

template <typename D>
void launch_act_grad(const void* dy, const void* z, int T, int O, int act, const BackPlan& p,
                     void* dz, float* sums, hipStream_t s) {
  typedef typename D::elem E;
  if (!sums) {
    const size_t chunks = static_cast<size_t>(T) * (O / D::V);
    hipLaunchKernelGGL(act_grad_kernel<D>, grid_of(chunks), dim3(256), 0, s,
                       static_cast<const E*>(dy), static_cast<const E*>(z), T, O, act,
                       static_cast<E*>(dz));
    return;
  }
  hipLaunchKernelGGL(act_grad_sum_kernel<D>, dim3((O + COLT * D::V - 1) / (COLT * D::V), p.blocks),
                     dim3(COLT * ROWT), 0, s, static_cast<const E*>(dy), static_cast<const E*>(z),
                     T, O, act, p.rows, static_cast<E*>(dz), sums);
}

template <bool PX, bool PW>
int launch_pair(const Mma& x, const Mma& w, const BiasSum& b, hipStream_t s) {
  constexpr int lds = (SA + SB) * 128 * SLICE * 2;
  const auto fn = mma_pair_kernel<PX, PW>;
  static std::atomic<bool> done[64];
  if (!allow_lds(reinterpret_cast<const void*>(fn), lds, done)) return MOE_EHIP;
  const int dw0 = grid_of(x), bias0 = dw0 + grid_of(w);
  hipLaunchKernelGGL(fn, dim3(bias0 + (b.dbias ? (b.W + 63) / 64 : 0)), dim3(W * MOE_WAVE), lds, s,
                     x, w, b, dw0, bias0);
  return MOE_OK;
}

// dx = dz w and dw = dz^T x (either may be absent: null y), and the bias's last
// sum where the two share a launch; b.dbias is cleared then.
inline int products(Mma x, Mma w, const BackPlan& p, BiasSum& b, float* part_x, float* part_w,
                    hipStream_t s) {
  if (!(p.pair && x.e.y && w.e.y)) {
    int rc = x.e.y ? product<false, true, false>(x, p.x, part_x, s) : MOE_OK;
    if (w.e.y && rc == MOE_OK) rc = product<true, true, false>(w, p.w, part_w, s);
    return rc;
  }
  cut(x, p.x, x.N, part_x);
  cut(w, p.w, w.N, part_w);
  const bool px = x.splits > 1, pw = w.splits > 1;
  const int rc = px ? (pw ? launch_pair<true, true>(x, w, b, s) : launch_pair<true, false>(x, w, b, s))
                    : (pw ? launch_pair<false, true>(x, w, b, s) : launch_pair<false, false>(x, w, b, s));
  b.dbias = nullptr;
  if (px && rc == MOE_OK) launch_join<uint16_t, false>(part_x, x.splits, x.M, x.N, x.e, s);
  if (pw && rc == MOE_OK) launch_join<uint16_t, false>(part_w, w.splits, w.M, w.N, w.e, s);
  return rc;
}

inline int products(const F32Prod& x, const F32Prod& w, const BackPlan& p, BiasSum& b,
                    float* part_x, float* part_w, hipStream_t s) {
  if (!(p.pair && x.e.y && w.e.y)) {
    int rc = x.e.y ? product_f32<false, true, false>(x, p.x, part_x, s) : MOE_OK;
    if (w.e.y && rc == MOE_OK) rc = product_f32<true, true, false>(w, p.w, part_w, s);
    return rc;
  }
  const int nx = (x.N + 31) / 32, dw0 = nx * ((x.M + 31) / 32), bias0 = dw0 + nx * ((w.M + 31) / 32);
  hipLaunchKernelGGL(f32_pair_kernel, dim3(bias0 + (b.dbias ? (b.W + 63) / 64 : 0)), dim3(256), 0, s,
                     x, w, b, nx, dw0, bias0);
  b.dbias = nullptr;
  return MOE_OK;
}

template <typename D, typename P>
int backward(const BackPlan& p, const void* dy, const void* x, const void* w, const void* z, int T,
             int K, int O, int act, void* dx, void* dw, void* dbias, char* ws, hipStream_t s) {
  typedef typename D::elem E;
  const int W = width(O, act);
  if (T == 0) {  // sums over no tokens
    if (!dw && !dbias) return MOE_OK;
    const size_t nw = static_cast<size_t>(W) * K;
    if (dw)
      hipLaunchKernelGGL(zero_kernel<E>, grid_of(nw), dim3(256), 0, s, static_cast<E*>(dw), nw);
    if (dbias)
      hipLaunchKernelGGL(zero_kernel<E>, grid_of(W), dim3(256), 0, s, static_cast<E*>(dbias),
                         static_cast<size_t>(W));
    return launch_status();
  }
  const void* dz = dy;
  BiasSum b{reinterpret_cast<float*>(ws + p.sums), p.blocks, W, dbias};
  if ((act != MOE_ACT_NONE && (dx || dw)) || dbias) {
    launch_act_grad<D>(dy, z, T, O, act, p, ws, dbias ? reinterpret_cast<float*>(ws + p.sums) : nullptr,
                       s);
    if (act != MOE_ACT_NONE) dz = ws;
  }
  P qx{};
  qx.r = static_cast<const E*>(dz);
  qx.ldr = W;
  qx.ldc = qx.N = K;
  P qw = qx;
  qx.c = static_cast<const E*>(w);
  qx.M = qw.K = T;
  qx.K = qw.M = W;
  qx.e.y = dx;
  qw.c = static_cast<const E*>(x);
  qw.e.y = dw;
  const int rc = products(qx, qw, p, b, reinterpret_cast<float*>(ws + p.part_x),
                          reinterpret_cast<float*>(ws + p.part_w), s);
  if (rc != MOE_OK) return rc;
  if (b.dbias) hipLaunchKernelGGL(bias_sum_kernel<E>, dim3((W + 63) / 64), dim3(256), 0, s, b);
  return launch_status();
}

}  // namespace lin
}  // namespace moe

using namespace moe;
using namespace moe::lin;

extern "C" size_t moe_linear_workspace_size(int T, int K, int O, int act, int dtype) {
  if (check(T, K, O, act, dtype) != MOE_OK) return 0;
  return forward_plan(T, K, O, act, dtype, cu_count()).bytes;
}

extern "C" int moe_linear(const void* x, const void* w, const void* bias, const void* residual,
                          int T, int K, int O, int act, int dtype, void* z, void* y,
                          void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check(T, K, O, act, dtype);
  if (rc != MOE_OK || T == 0) return rc;
  if (!x || !w || !y || !workspace) return MOE_EINVAL;
  for (const void* q : {x, w, bias, residual, static_cast<const void*>(z),
                        static_cast<const void*>(y), static_cast<const void*>(workspace)})
    if (!aligned16(q)) return MOE_EINVAL;
  const ForwardPlan f = forward_plan(T, K, O, act, dtype, cu_count());
  if (workspace_bytes < f.bytes) return MOE_EINVAL;
  hipStream_t s = as_stream(stream);
  const bool glu = act == MOE_ACT_SWIGLU;
  const Epilogue e{bias, residual, z, y, act};
  float* part = static_cast<float*>(workspace);
  int r;
  if (f.rf) {
    const Skinny q{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w), T, K, O, 0, 0, e};
    r = glu ? launch_skinny<true>(q, f.rf, s) : launch_skinny<false>(q, f.rf, s);
  } else if (dtype == MOE_BF16) {
    Mma q{};
    q.r = static_cast<const uint16_t*>(x);
    q.c = static_cast<const uint16_t*>(w);
    q.ldr = q.ldc = K;
    q.M = T;
    q.N = O;
    q.K = K;
    q.e = e;
    r = glu ? product<false, false, true>(q, f.p, part, s)
            : product<false, false, false>(q, f.p, part, s);
  } else {
    F32Prod q{};
    q.r = static_cast<const float*>(x);
    q.c = static_cast<const float*>(w);
    q.ldr = q.ldc = K;
    q.M = T;
    q.N = O;
    q.K = K;
    q.e = e;
    r = glu ? product_f32<false, false, true>(q, f.p, part, s)
            : product_f32<false, false, false>(q, f.p, part, s);
  }
  return r == MOE_OK ? launch_status() : r;
}

extern "C" size_t moe_linear_backward_workspace_size(int T, int K, int O, int act, int dtype) {
  if (check(T, K, O, act, dtype) != MOE_OK) return 0;
  return back_plan(T, K, O, act, dtype, cu_count()).bytes;
}

extern "C" int moe_linear_backward(const void* dy, const void* x, const void* w, const void* z,
                                   int T, int K, int O, int act, int dtype, void* dx, void* dw,
                                   void* dbias, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  const int rc = check(T, K, O, act, dtype);
  if (rc != MOE_OK) return rc;
  if (T > 0 && ((!dx && !dw && !dbias) || !dy || (act != MOE_ACT_NONE && !z) || (dx && !w) ||
                (dw && !x) || !workspace))
    return MOE_EINVAL;  // without tokens dx is empty and its address may be null
  for (const void* q : {dy, x, w, z, static_cast<const void*>(dx), static_cast<const void*>(dw),
                        static_cast<const void*>(dbias), static_cast<const void*>(workspace)})
    if (!aligned16(q)) return MOE_EINVAL;
  const BackPlan p = back_plan(T, K, O, act, dtype, cu_count());
  if (T > 0 && workspace_bytes < p.bytes) return MOE_EINVAL;
  char* ws = static_cast<char*>(workspace);
  hipStream_t s = as_stream(stream);
  if (dtype == MOE_BF16)
    return backward<Bf16, Mma>(p, dy, x, w, z, T, K, O, act, dx, dw, dbias, ws, s);
  return backward<F32, F32Prod>(p, dy, x, w, z, T, K, O, act, dx, dw, dbias, ws, s);
}
