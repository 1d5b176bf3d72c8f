// moe_linear and moe_linear_backward: the matrix product of the dense parts
// beside the routed experts, with bias, activation and residual in its
// epilogue, and its gradients.
//
//   z = x W^T + b,   y = act(z) + residual
//   dz = dy act'(z);   dx = dz W,   dW = dz^T x,   db = sum_t dz
//
// act "swiglu" takes W [2O,K], gate rows first: y = silu(z[:, :O]) z[:, O:].
#include <algorithm>
#include <type_traits>

#include "common.h"

namespace moe {
namespace lin {

typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float load_elem(const float* p) { return *p; }
__device__ __forceinline__ float load_elem(const __bf16* p) { return static_cast<float>(*p); }
__device__ __forceinline__ void store_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_elem(__bf16* p, float v) { *p = static_cast<__bf16>(v); }

// ------------------------------------------------------------- activations
__device__ __forceinline__ float sigmoid(float a) { return 1.f / (1.f + expf(-a)); }
__device__ __forceinline__ float gauss_cdf(float a) {
  return 0.5f * erfcf(a * -0.70710678118654752f);
}

__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? z : 0.f;
    case MOE_ACT_SILU: return z * sigmoid(z);
    case MOE_ACT_GELU: return z * gauss_cdf(z);
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(int act, float z) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case MOE_ACT_SILU: {
      const float s = sigmoid(z);
      return s * (1.f + z * (1.f - s));
    }
    case MOE_ACT_GELU: return gauss_cdf(z) + z * 0.39894228040143268f * expf(-0.5f * z * z);
    default: return 1.f;
  }
}

// ------------------------------------------------------------ tile product
// C[m][n] = sum_k A(m, k) B(n, k), A(m, k) = a[m * am + k * ak] and so on.
struct Prod {
  const void *a, *b;
  long am, ak, bm, bk;
  int M, N, K;
  // epilogue
  int act;
  const void *bias, *residual;
  void *z, *c;
};

constexpr int TILE = 64, BK = 16, NTHR = 256;

template <typename E, bool GLU>
__global__ __launch_bounds__(NTHR) void product_kernel(Prod p) {
  __shared__ float sa[BK][TILE + 1], sb[GLU ? 2 : 1][BK][TILE + 1];
  const E* a = static_cast<const E*>(p.a);
  const E* b = static_cast<const E*>(p.b);
  const int m0 = blockIdx.y * TILE, n0 = blockIdx.x * TILE;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[GLU ? 2 : 1][4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += BK) {
    __syncthreads();
    for (int i = threadIdx.x; i < TILE * BK; i += NTHR) {
      // consecutive threads along the operand's contiguous axis
      const int am = p.ak == 1 ? i / BK : i % TILE, ak = p.ak == 1 ? i % BK : i / TILE;
      const int bm = p.bk == 1 ? i / BK : i % TILE, bk = p.bk == 1 ? i % BK : i / TILE;
      sa[ak][am] = m0 + am < p.M && k0 + ak < p.K ? load_elem(a + (m0 + am) * p.am + (k0 + ak) * p.ak)
                                                  : 0.f;
#pragma unroll
      for (int h = 0; h < (GLU ? 2 : 1); ++h)
        sb[h][bk][bm] = n0 + bm < p.N && k0 + bk < p.K
                            ? load_elem(b + (h * static_cast<long>(p.N) + n0 + bm) * p.bm + (k0 + bk) * p.bk)
                            : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < BK; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int h = 0; h < (GLU ? 2 : 1); ++h)
            acc[h][i][j] += sa[kk][ty * 4 + i] * sb[h][kk][tx * 4 + j];
  }
  const E* bias = static_cast<const E*>(p.bias);
  const E* residual = static_cast<const E*>(p.residual);
  E* z = static_cast<E*>(p.z);
  E* c = static_cast<E*>(p.c);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= p.M || n >= p.N) continue;
      const size_t at = static_cast<size_t>(m) * p.N + n;
      float v;
      if constexpr (GLU) {
        const float g = acc[0][i][j] + (bias ? load_elem(bias + n) : 0.f);
        const float u = acc[1][i][j] + (bias ? load_elem(bias + p.N + n) : 0.f);
        if (z) {
          const size_t zr = static_cast<size_t>(m) * 2 * p.N;
          store_elem(z + zr + n, g);
          store_elem(z + zr + p.N + n, u);
        }
        v = g * sigmoid(g) * u;
      } else {
        const float s = acc[0][i][j] + (bias ? load_elem(bias + n) : 0.f);
        if (z) store_elem(z + at, s);
        v = act_value(p.act, s);
      }
      if (residual) v += load_elem(residual + at);
      store_elem(c + at, v);
    }
}

template <typename E>
void launch_product(const Prod& p, bool glu, hipStream_t s) {
  const dim3 grid((p.N + TILE - 1) / TILE, (p.M + TILE - 1) / TILE);
  if (glu) hipLaunchKernelGGL((product_kernel<E, true>), grid, dim3(NTHR), 0, s, p);
  else hipLaunchKernelGGL((product_kernel<E, false>), grid, dim3(NTHR), 0, s, p);
}

// ------------------------------------------------ activation gradient, bias
// dz (rounded to the element type, the operand of both products) and, per
// block of token rows, the fp32 column sums of the unrounded dz.
constexpr int ROWS = 64;

template <typename E>
__global__ __launch_bounds__(64) void act_grad_kernel(const E* __restrict__ dy,
                                                      const E* __restrict__ z, int T, int O,
                                                      int act, E* __restrict__ dz,
                                                      float* __restrict__ part) {
  const int o = blockIdx.x * 64 + threadIdx.x;
  if (o >= O) return;
  const int W = act == MOE_ACT_SWIGLU ? 2 * O : O;
  float s0 = 0.f, s1 = 0.f;
  const int t1 = min(T, static_cast<int>(blockIdx.y + 1) * ROWS);
  for (int t = blockIdx.y * ROWS; t < t1; ++t) {
    const float g = load_elem(dy + static_cast<size_t>(t) * O + o);
    const size_t zr = static_cast<size_t>(t) * W + o;
    if (act == MOE_ACT_SWIGLU) {
      const float a = load_elem(z + zr), b = load_elem(z + zr + O);
      const float da = g * b * act_slope(MOE_ACT_SILU, a), db = g * a * sigmoid(a);
      store_elem(dz + zr, da);
      store_elem(dz + zr + O, db);
      s0 += da;
      s1 += db;
    } else {
      const float d = act == MOE_ACT_NONE ? g : g * act_slope(act, load_elem(z + zr));
      if (act != MOE_ACT_NONE) store_elem(dz + zr, d);
      s0 += d;
    }
  }
  if (part) {
    part[static_cast<size_t>(blockIdx.y) * W + o] = s0;
    if (act == MOE_ACT_SWIGLU) part[static_cast<size_t>(blockIdx.y) * W + O + o] = s1;
  }
}

template <typename E>
__global__ __launch_bounds__(64) void bias_sum_kernel(const float* __restrict__ part, int blocks,
                                                      int W, E* __restrict__ dbias) {
  const int o = blockIdx.x * 64 + threadIdx.x;
  if (o >= W) return;
  float s = 0.f;
  for (int b = 0; b < blocks; ++b) s += part[static_cast<size_t>(b) * W + o];
  store_elem(dbias + o, s);
}

template <typename E>
__global__ void zero_kernel(E* p, size_t n) {
  const size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x;
  if (i < n) store_elem(p + i, 0.f);
}

// --------------------------------------------------------------------- host
inline size_t elem_size(int dtype) { return dtype == MOE_BF16 ? 2 : 4; }
inline size_t up256(size_t n) { return (n + 255) & ~size_t(255); }
inline int width(int O, int act) { return act == MOE_ACT_SWIGLU ? 2 * O : O; }
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

struct BackPlan {
  size_t dz, part, bytes;  // offsets, size
  int blocks;
};

inline BackPlan back_plan(int T, int O, int act, int dtype) {
  BackPlan p;
  const size_t W = width(O, act);
  p.blocks = (T + ROWS - 1) / ROWS;
  p.dz = 0;
  p.part = act == MOE_ACT_NONE ? 0 : up256(static_cast<size_t>(T) * W * elem_size(dtype));
  p.bytes = p.part + up256(static_cast<size_t>(p.blocks) * W * 4) + 256;
  return p;
}

template <typename E>
int backward(const void* dy, const void* x, const void* w, const void* z, int T, int K, int O,
             int act, int dtype, void* dx, void* dw, void* dbias, char* ws, hipStream_t s) {
  const BackPlan p = back_plan(T, O, act, dtype);
  const int W = width(O, act);
  if (T == 0) {  // sums over no tokens
    if (!dw && !dbias) return MOE_OK;
    const size_t nw = static_cast<size_t>(W) * K;
    if (dw)
      hipLaunchKernelGGL(zero_kernel<E>, dim3((nw + 255) / 256), dim3(256), 0, s,
                         static_cast<E*>(dw), nw);
    if (dbias)
      hipLaunchKernelGGL(zero_kernel<E>, dim3((W + 255) / 256), dim3(256), 0, s,
                         static_cast<E*>(dbias), static_cast<size_t>(W));
    return launch_status();
  }
  const void* dz = dy;
  float* part = dbias ? reinterpret_cast<float*>(ws + p.part) : nullptr;
  if (act != MOE_ACT_NONE || dbias) {
    hipLaunchKernelGGL(act_grad_kernel<E>, dim3((O + 63) / 64, p.blocks), dim3(64), 0, s,
                       static_cast<const E*>(dy), static_cast<const E*>(z), T, O, act,
                       reinterpret_cast<E*>(ws + p.dz), part);
    if (act != MOE_ACT_NONE) dz = ws + p.dz;
  }
  if (dbias)
    hipLaunchKernelGGL(bias_sum_kernel<E>, dim3((W + 63) / 64), dim3(64), 0, s, part, p.blocks, W,
                       static_cast<E*>(dbias));
  if (dx) {
    Prod q{};
    q.a = dz; q.am = W; q.ak = 1;
    q.b = w; q.bm = 1; q.bk = K;
    q.M = T; q.N = K; q.K = W;
    q.c = dx;
    launch_product<E>(q, false, s);
  }
  if (dw) {
    Prod q{};
    q.a = dz; q.am = 1; q.ak = W;
    q.b = x; q.bm = 1; q.bk = K;
    q.M = W; q.N = K; q.K = T;
    q.c = dw;
    launch_product<E>(q, false, s);
  }
  return launch_status();
}

}  // namespace lin
}  // namespace moe

using namespace moe;
using namespace moe::lin;

extern "C" size_t moe_linear_workspace_size(int T, int K, int O, int act, int dtype) {
  if (check(T, K, O, act, dtype) != MOE_OK) return 0;
  return 256;
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
  if (workspace_bytes < moe_linear_workspace_size(T, K, O, act, dtype)) return MOE_EINVAL;
  hipStream_t s = as_stream(stream);
  Prod p{};
  p.a = x; p.am = K; p.ak = 1;
  p.b = w; p.bm = K; p.bk = 1;
  p.M = T; p.N = O; p.K = K;
  p.act = act;
  p.bias = bias; p.residual = residual;
  p.z = z; p.c = y;
  if (dtype == MOE_BF16) launch_product<__bf16>(p, act == MOE_ACT_SWIGLU, s);
  else launch_product<float>(p, act == MOE_ACT_SWIGLU, s);
  return launch_status();
}

extern "C" size_t moe_linear_backward_workspace_size(int T, int K, int O, int act, int dtype) {
  if (check(T, K, O, act, dtype) != MOE_OK) return 0;
  return back_plan(T, O, act, dtype).bytes;
}

extern "C" int moe_linear_backward(const void* dy, const void* x, const void* w, const void* z,
                                   int T, int K, int O, int act, int dtype, void* dx, void* dw,
                                   void* dbias, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  const int rc = check(T, K, O, act, dtype);
  if (rc != MOE_OK) return rc;
  if (!dx && !dw && !dbias) return MOE_EINVAL;
  if (T > 0 && (!dy || (act != MOE_ACT_NONE && !z) || (dx && !w) || (dw && !x) || !workspace))
    return MOE_EINVAL;
  for (const void* q : {dy, x, w, z, static_cast<const void*>(dx), static_cast<const void*>(dw),
                        static_cast<const void*>(dbias), static_cast<const void*>(workspace)})
    if (!aligned16(q)) return MOE_EINVAL;
  if (T > 0 && workspace_bytes < moe_linear_backward_workspace_size(T, K, O, act, dtype))
    return MOE_EINVAL;
  char* ws = static_cast<char*>(workspace);
  hipStream_t s = as_stream(stream);
  if (dtype == MOE_BF16)
    return backward<__bf16>(dy, x, w, z, T, K, O, act, dtype, dx, dw, dbias, ws, s);
  return backward<float>(dy, x, w, z, T, K, O, act, dtype, dx, dw, dbias, ws, s);
}
