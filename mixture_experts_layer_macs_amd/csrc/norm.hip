// moe_norm and moe_norm_backward: layer norm (or rms: mean = 0) of the residual
// sum, and its gradients.
//
//   s = x + residual;  h = (s - mean) rstd;  y = h w + b
//   u = dy w;  dx = rstd (u - mean(u) - h mean(u h)) + dsum
//   dw = sum_t dy h;  db = sum_t dy
//
// Bound by HBM: every array is read or written once.  A row lives in the
// registers of TPR threads, 16 bytes a time and thread, so that the variance is
// taken from centred values without a second read; rows too wide for that are
// read again, from L2.  s is rounded to the element type before it is
// normalised: the backward pass and the rest of the layer see that value.
//
// Measured: 8192 x 2048 bf16 rms with residual 22 us forward (134 MB, 6.1 TB/s with
// inputs in the last-level cache), 31 backward (134 MB, 4.3 TB/s) and 4 to join the
// column sums; 16381 x 1028 fp32 24, 41 (5.0 TB/s) and 4; one row 3.8, latency.  Wide
// rows: 2048 x 16384 with bias 28 forward and 94 backward in bf16, 70 and 172 in fp32.
#include <algorithm>

#include "common.h"
#include "linear_common.h"

namespace moe {
namespace norm {

using lin::aligned16;
using lin::Bf16;
using lin::F32;
using lin::load_v;
using lin::store1;
using lin::store_v;

struct Forward {
  const void *x, *residual, *weight, *bias;
  int T, H;
  bool rms;
  float eps;
  void *sum, *y;
  float *mean, *rstd;
};

struct Backward {
  const void *dy, *s, *weight;
  const float *mean, *rstd;  // mean: null for rms
  const void* dsum;
  int T, H;
  void *dx, *dweight, *dbias;
  float* part;  // [blocks][2][H] sums of the workgroups; null: one workgroup, written as they are
};

// Sum over the TPR threads of a row.  Rows wider than a wave go through LDS, in
// two places in turn, so that one barrier a sum is enough.
template <int TPR>
struct RowSum {
  float (*red)[TPR / MOE_WAVE > 0 ? TPR / MOE_WAVE : 1];
  int turn = 0;
  __device__ __forceinline__ float operator()(float v) {
    if constexpr (TPR == 16) {
      v += dpp_t<float, DPP_QUAD_1032>(0.f, v);
      v += dpp_t<float, DPP_QUAD_2301>(0.f, v);
      v += dpp_t<float, DPP_ROW_HALF_MIRROR>(0.f, v);
      v += dpp_t<float, 0x140>(0.f, v);  // lane 15-i of each row
      return v;
    } else {
      v = wave_sum(v);
      if constexpr (TPR > MOE_WAVE) {
        float* r = red[turn];
        turn ^= 1;
        if (lane_id() == 0) r[threadIdx.x / MOE_WAVE] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / MOE_WAVE; ++i) v += r[i];
      }
      return v;
    }
  }
};

constexpr int threads_of(int tpr) { return tpr > 256 ? tpr : 256; }
// Backward: 8 waves, so that few workgroups leave few column sums to join.
constexpr int back_threads_of(int tpr) { return tpr > 64 ? tpr : 512; }

// 16 bytes of an array, or zeros
template <typename E, int V>
__device__ __forceinline__ void load_if(const E* p, bool in, float* f) {
  if (in) {
    load_v<V>(p, f);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = 0.f;
  }
}

// v as it is read back from the element type
__device__ __forceinline__ float rounded(float v, const uint16_t*) {
  return static_cast<float>(static_cast<__bf16>(v));
}
__device__ __forceinline__ float rounded(float v, const float*) { return v; }

template <typename E, int V>
__device__ __forceinline__ void norm_out(const Forward& a, size_t row, int col, const float* s,
                                         float mean, float rstd) {
  float w[V], b[V], y[V];
  load_v<V>(static_cast<const E*>(a.weight) + col, w);
#pragma unroll
  for (int i = 0; i < V; ++i) y[i] = (s[i] - mean) * rstd * w[i];
  if (a.bias) {
    load_v<V>(static_cast<const E*>(a.bias) + col, b);
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] += b[i];
  }
  store_v<V>(static_cast<E*>(a.y) + row + col, y);
}

template <typename E, int V>
__device__ __forceinline__ void sum_in(const Forward& a, size_t row, int col, float* s) {
  load_v<V>(static_cast<const E*>(a.x) + row + col, s);
  if (a.residual) {
    float r[V];
    load_v<V>(static_cast<const E*>(a.residual) + row + col, r);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = rounded(s[i] + r[i], static_cast<const E*>(nullptr));
    store_v<V>(static_cast<E*>(a.sum) + row + col, s);
  }
}

template <typename D, int TPR, int NV>
__global__ __launch_bounds__(threads_of(TPR)) void norm_kernel(Forward a) {
  typedef typename D::elem E;
  constexpr int V = D::V, ROWS = threads_of(TPR) / TPR;
  __shared__ float red[2][TPR / MOE_WAVE > 0 ? TPR / MOE_WAVE : 1];
  RowSum<TPR> sum{red};
  const int l = threadIdx.x % TPR, t = blockIdx.x * ROWS + threadIdx.x / TPR;
  if (t >= a.T) return;  // whole rows of lanes; TPR > 64: one row per workgroup, never
  const size_t row = static_cast<size_t>(t) * a.H;
  float s[NV][V], total = 0.f, square = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = (l + TPR * j) * V;
    if (col < a.H) {
      sum_in<E, V>(a, row, col, s[j]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) s[j][i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) total += s[j][i];
  }
  const float mean = a.rms ? 0.f : sum(total) / a.H;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if ((l + TPR * j) * V < a.H)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float c = s[j][i] - mean;
        square += c * c;
      }
  const float rstd = 1.f / sqrtf(sum(square) / a.H + a.eps);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = (l + TPR * j) * V;
    if (col < a.H) norm_out<E, V>(a, row, col, s[j], mean, rstd);
  }
  if (l == 0) {
    if (a.mean) a.mean[t] = mean;
    if (a.rstd) a.rstd[t] = rstd;
  }
}

// Rows of more columns than the registers of a workgroup hold at a time: the
// sum is read back from where it was stored, each thread its own elements.
constexpr int WIDE = 1024;

template <typename D>
__global__ __launch_bounds__(WIDE) void norm_wide_kernel(Forward a) {
  typedef typename D::elem E;
  constexpr int V = D::V;
  __shared__ float red[2][WIDE / MOE_WAVE];
  RowSum<WIDE> sum{red};
  const int t = blockIdx.x, l = threadIdx.x;
  const size_t row = static_cast<size_t>(t) * a.H;
  const E* src = static_cast<const E*>(a.residual ? a.sum : a.x) + row;
  float s[V], total = 0.f, square = 0.f;
  for (int col = l * V; col < a.H; col += WIDE * V) {
    sum_in<E, V>(a, row, col, s);
#pragma unroll
    for (int i = 0; i < V; ++i) total += s[i];
  }
  const float mean = a.rms ? 0.f : sum(total) / a.H;
  for (int col = l * V; col < a.H; col += WIDE * V) {
    load_v<V>(src + col, s);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float c = s[i] - mean;
      square += c * c;
    }
  }
  const float rstd = 1.f / sqrtf(sum(square) / a.H + a.eps);
  for (int col = l * V; col < a.H; col += WIDE * V) {
    load_v<V>(src + col, s);
    norm_out<E, V>(a, row, col, s, mean, rstd);
  }
  if (l == 0) {
    if (a.mean) a.mean[t] = mean;
    if (a.rstd) a.rstd[t] = rstd;
  }
}

// ------------------------------------------------------------------ backward
// 16 bytes as they lie in memory, and their values
template <int V>
__device__ __forceinline__ void values(lin::u32x4 w, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (V == 8) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      f[i] = __uint_as_float(w[i]);
    }
  }
}

// The workgroup's sums of V columns
template <typename E, int V>
__device__ __forceinline__ void sums_out(const Backward& a, int col, const float* w, const float* b) {
  if (a.part) {
    float* p = a.part + static_cast<size_t>(blockIdx.x) * 2 * a.H + col;
    store_v<V>(p, w);
    store_v<V>(p + a.H, b);
    return;
  }
  if (a.dweight) store_v<V>(static_cast<E*>(a.dweight) + col, w);
  if (a.dbias) store_v<V>(static_cast<E*>(a.dbias) + col, b);
}

// A group of TPR threads takes every (workgroups x ROWS)-th row, the next one's
// arrays in flight while one is worked on, and keeps the column sums of its rows
// in registers; the workgroup's groups add theirs in order through LDS.
// BIAS: the bias's column sums are wanted (their registers otherwise are not).
template <typename D, int TPR, int NV, bool BIAS>
__global__ __launch_bounds__(back_threads_of(TPR)) void norm_backward_kernel(Backward a) {
  typedef typename D::elem E;
  constexpr int V = D::V, ROWS = back_threads_of(TPR) / TPR;
  __shared__ float red[2][TPR / MOE_WAVE > 0 ? TPR / MOE_WAVE : 1];
  __shared__ float cols[2][ROWS > 1 ? TPR * NV * V : 1];
  RowSum<TPR> sum{red};
  const int l = threadIdx.x % TPR, group = threadIdx.x / TPR;
  lin::u32x4 dyn[NV], sn[NV], gn[NV];
  float mean_n = 0.f, rstd_n;
  auto piece = [&](const void* p, size_t row, int j) {
    const int col = (l + TPR * j) * V;
    const size_t at = row + (col < a.H ? col : 0);  // past the end: a piece that is not used
    return *reinterpret_cast<const lin::u32x4*>(static_cast<const E*>(p) + at);
  };
  auto row_of = [&](int t) { return static_cast<size_t>(min(t, a.T - 1)) * a.H; };
  auto request = [&](int t) {
    const size_t row = row_of(t);
    t = min(t, a.T - 1);
    if (a.mean) mean_n = a.mean[t];
    rstd_n = a.rstd[t];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      dyn[j] = piece(a.dy, row, j);
      sn[j] = piece(a.s, row, j);
    }
  };
  auto request_sum = [&](int t) {
    const size_t row = row_of(t);
#pragma unroll
    for (int j = 0; j < NV; ++j) gn[j] = a.dsum ? piece(a.dsum, row, j) : lin::u32x4{0, 0, 0, 0};
  };
  float aw[NV][V] = {}, ab[NV][V] = {};
  int t = blockIdx.x * ROWS + group;
  request(t);
  request_sum(t);
  for (; t < a.T; t += gridDim.x * ROWS) {
    const size_t row = static_cast<size_t>(t) * a.H;
    const float mean = mean_n, rstd = rstd_n;
    float h[NV][V], u = 0.f, uh = 0.f;
    lin::u32x4 dyr[NV];  // as it lies: half the registers of its values in bf16
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = (l + TPR * j) * V < a.H;
      dyr[j] = in ? dyn[j] : lin::u32x4{0, 0, 0, 0};
      values<V>(sn[j], h[j]);
#pragma unroll
      for (int i = 0; i < V; ++i) h[j][i] = in ? (h[j][i] - mean) * rstd : 0.f;
    }
    request(t + gridDim.x * ROWS);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float dy[V], w[V] = {};
      values<V>(dyr[j], dy);
      if (a.dx) values<V>(piece(a.weight, 0, j), w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        aw[j][i] += dy[i] * h[j][i];
        if constexpr (BIAS) ab[j][i] += dy[i];
        u += dy[i] * w[i];
        uh += dy[i] * w[i] * h[j][i];
      }
    }
    if (!a.dx) continue;
    const float mu = a.mean ? sum(u) / a.H : 0.f, muh = sum(uh) / a.H;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (l + TPR * j) * V;
      float dy[V], w[V], g[V];
      values<V>(dyr[j], dy);
      values<V>(piece(a.weight, 0, j), w);
      values<V>(gn[j], g);
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] += rstd * (dy[i] * w[i] - mu - h[j][i] * muh);
      if (col < a.H) store_v<V>(static_cast<E*>(a.dx) + row + col, g);
    }
    request_sum(t + gridDim.x * ROWS);
  }
  if (!a.dweight && !a.dbias) return;
  if constexpr (ROWS == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (l + TPR * j) * V;
      if (col < a.H) sums_out<E, V>(a, col, aw[j], ab[j]);
    }
  } else {
    for (int g = 0; g < ROWS; ++g) {
      if (g == group)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int c = (l + TPR * j) * V + i;
            cols[0][c] = g ? cols[0][c] + aw[j][i] : aw[j][i];
            cols[1][c] = g ? cols[1][c] + ab[j][i] : ab[j][i];
          }
      __syncthreads();
    }
    for (int c = threadIdx.x * V; c < a.H; c += back_threads_of(TPR) * V)
      sums_out<E, V>(a, c, cols[0] + c, cols[1] + c);
  }
}

// Wide rows: dx alone, the row read a second time from L2 ...
template <typename D>
__global__ __launch_bounds__(WIDE) void norm_backward_wide_kernel(Backward a) {
  typedef typename D::elem E;
  constexpr int V = D::V;
  __shared__ float red[2][WIDE / MOE_WAVE];
  RowSum<WIDE> sum{red};
  const int t = blockIdx.x, l = threadIdx.x;
  const size_t row = static_cast<size_t>(t) * a.H;
  const float mean = a.mean ? a.mean[t] : 0.f, rstd = a.rstd[t];
  const E *pdy = static_cast<const E*>(a.dy) + row, *ps = static_cast<const E*>(a.s) + row;
  float dy[V], h[V], w[V], g[V], u = 0.f, uh = 0.f;
  for (int col = l * V; col < a.H; col += WIDE * V) {
    load_v<V>(pdy + col, dy);
    load_v<V>(ps + col, h);
    load_v<V>(static_cast<const E*>(a.weight) + col, w);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      u += dy[i] * w[i];
      uh += dy[i] * w[i] * ((h[i] - mean) * rstd);
    }
  }
  const float mu = a.mean ? sum(u) / a.H : 0.f, muh = sum(uh) / a.H;
  for (int col = l * V; col < a.H; col += WIDE * V) {
    load_v<V>(pdy + col, dy);
    load_v<V>(ps + col, h);
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = (h[i] - mean) * rstd;
    load_v<V>(static_cast<const E*>(a.weight) + col, w);
    load_if<E, V>(static_cast<const E*>(a.dsum) + row + col, a.dsum != nullptr, g);
#pragma unroll
    for (int i = 0; i < V; ++i) dy[i] = rstd * (dy[i] * w[i] - mu - h[i] * muh) + g[i];
    store_v<V>(static_cast<E*>(a.dx) + row + col, dy);
  }
}

// ... and the column sums before it (dx may take dy's place): a thread owns 16
// bytes of columns in every gridDim.y-th row.
template <typename D>
__global__ __launch_bounds__(256) void norm_columns_kernel(Backward a) {
  typedef typename D::elem E;
  constexpr int V = D::V;
  const int col = (blockIdx.x * 256 + threadIdx.x) * V;
  if (col >= a.H) return;
  float aw[V] = {}, ab[V] = {};
  for (int t = blockIdx.y; t < a.T; t += gridDim.y) {
    const size_t at = static_cast<size_t>(t) * a.H + col;
    const float mean = a.mean ? a.mean[t] : 0.f, rstd = a.rstd[t];
    float dy[V], h[V];
    load_v<V>(static_cast<const E*>(a.dy) + at, dy);
    load_v<V>(static_cast<const E*>(a.s) + at, h);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      aw[i] += dy[i] * ((h[i] - mean) * rstd);
      ab[i] += dy[i];
    }
  }
  float* p = a.part + static_cast<size_t>(blockIdx.y) * 2 * a.H + col;
  store_v<V>(p, aw);
  store_v<V>(p + a.H, ab);
}

// The workgroups' sums to the outputs, in their order: 64 columns a workgroup,
// 16 threads to a column.  blockIdx.y 0: dweight, 1: dbias.
template <typename E>
__global__ __launch_bounds__(1024) void norm_join_kernel(const float* __restrict__ part, int blocks,
                                                         int H, void* dweight, void* dbias) {
  __shared__ double red[16][64];
  void* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  const int c = threadIdx.x % 64, r = threadIdx.x / 64, col = blockIdx.x * 64 + c;
  double v = 0.0;
  if (col < H) {
    const float* p = part + blockIdx.y * static_cast<size_t>(H) + col;
#pragma unroll 8
    for (int i = r; i < blocks; i += 16) v += static_cast<double>(p[static_cast<size_t>(i) * 2 * H]);
  }
  red[r][c] = v;
  __syncthreads();
  if (r == 0 && col < H) {
    for (int i = 1; i < 16; ++i) v += red[i][c];
    store1(static_cast<E*>(out) + col, static_cast<float>(v));
  }
}

// --------------------------------------------------------------------- host
struct Shape {
  int tpr, nv;  // tpr 0: wide rows
};

// Threads of a row and 16-byte pieces of each: a wave while its lanes hold at
// most 32 columns (the backward pass keeps six values per column), else four
// waves.  (fp32 rows of 1028 in four waves, the second piece all but empty: 57 us
// backward for 16381 rows.)  bf16 rows of 1544 to 2048 columns with both column
// sums do not fit: the backward kernel spills 6 of 256 registers to scratch memory in
// its loop (8192 x 2048 layer norm: 31.7 us, 31.0 without bias, which spills none).
inline Shape shape_of(int H, int dtype) {
  const int most = dtype == MOE_BF16 ? 4 : 6, pieces = H / (dtype == MOE_BF16 ? 8 : 4);
  if (pieces <= 16) return {16, 1};
  const int tpr = pieces <= 64 * most ? 64 : 256, nv = (pieces + tpr - 1) / tpr;
  if (nv > most) return {0, 0};
  return {tpr, nv};
}

// Workgroups that keep column sums: 8 waves to a CU.
inline int sum_blocks(int T, int H, int dtype) {
  const Shape s = shape_of(H, dtype);
  const int rows = s.tpr ? back_threads_of(s.tpr) / s.tpr : 1;
  return std::max(1, std::min((T + rows - 1) / rows, s.tpr && s.tpr < 256 ? cu_count() : 2 * cu_count()));
}

inline int check(int T, int H, int kind, int dtype) {
  if (T < 0 || T > (1 << 20) || H < 1 || H > MOE_LINEAR_MAX_DIM ||
      (kind != MOE_NORM_LAYER && kind != MOE_NORM_RMS))
    return MOE_EINVAL;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EUNSUP;
  return H % (dtype == MOE_BF16 ? 8 : 4) ? MOE_EUNSUP : MOE_OK;
}

template <typename D, int TPR, int NV>
void launch(const Forward& a, hipStream_t s) {
  constexpr int rows = threads_of(TPR) / TPR;
  hipLaunchKernelGGL((norm_kernel<D, TPR, NV>), dim3((a.T + rows - 1) / rows),
                     dim3(threads_of(TPR)), 0, s, a);
}
template <typename D, int TPR, int NV>
void launch(const Backward& a, hipStream_t s, int blocks) {
  const dim3 block(back_threads_of(TPR));
  if (a.dbias)
    hipLaunchKernelGGL((norm_backward_kernel<D, TPR, NV, true>), dim3(blocks), block, 0, s, a);
  else
    hipLaunchKernelGGL((norm_backward_kernel<D, TPR, NV, false>), dim3(blocks), block, 0, s, a);
}

template <typename D, int TPR, typename A, typename... Rest>
void launch_pieces(int nv, const A& a, Rest... rest) {
  switch (nv) {
    case 1: return launch<D, TPR, 1>(a, rest...);
    case 2: return launch<D, TPR, 2>(a, rest...);
    case 3: return launch<D, TPR, 3>(a, rest...);
    case 4: return launch<D, TPR, 4>(a, rest...);
  }
  if constexpr (D::V == 4) {
    if (nv == 5) launch<D, TPR, 5>(a, rest...);
    else launch<D, TPR, 6>(a, rest...);
  }
}

template <typename D, typename A, typename... Rest>
void launch_shape(Shape p, const A& a, Rest... rest) {
  if (p.tpr == 16) launch<D, 16, 1>(a, rest...);
  else if (p.tpr == 64) launch_pieces<D, 64>(p.nv, a, rest...);
  else launch_pieces<D, 256>(p.nv, a, rest...);
}

template <typename D>
int forward(const Forward& a, int dtype, hipStream_t s) {
  const Shape p = shape_of(a.H, dtype);
  if (p.tpr) launch_shape<D>(p, a, s);
  else hipLaunchKernelGGL(norm_wide_kernel<D>, dim3(a.T), dim3(WIDE), 0, s, a);
  return launch_status();
}

template <typename D>
int backward(Backward a, int dtype, float* ws, hipStream_t s) {
  typedef typename D::elem E;
  const bool sums = a.dweight || a.dbias;
  if (a.T == 0) {  // sums over no tokens
    if (!sums) return MOE_OK;
    for (void* p : {a.dweight, a.dbias})
      if (p)
        hipLaunchKernelGGL(lin::zero_kernel<E>, dim3((a.H + 255) / 256), dim3(256), 0, s,
                           static_cast<E*>(p), static_cast<size_t>(a.H));
    return launch_status();
  }
  const Shape p = shape_of(a.H, dtype);
  const int blocks = sum_blocks(a.T, a.H, dtype);
  a.part = blocks > 1 || !p.tpr ? ws : nullptr;
  if (p.tpr) {
    launch_shape<D>(p, a, s, blocks);
  } else {
    if (sums)
      hipLaunchKernelGGL(norm_columns_kernel<D>, dim3((a.H / D::V + 255) / 256, blocks), dim3(256), 0,
                         s, a);
    if (a.dx) hipLaunchKernelGGL(norm_backward_wide_kernel<D>, dim3(a.T), dim3(WIDE), 0, s, a);
  }
  if (sums && a.part)
    hipLaunchKernelGGL(norm_join_kernel<E>, dim3((a.H + 63) / 64, 2), dim3(1024), 0, s, a.part,
                       blocks, a.H, a.dweight, a.dbias);
  return launch_status();
}

}  // namespace norm
}  // namespace moe

using namespace moe;
using namespace moe::norm;

extern "C" int moe_norm(const void* x, const void* residual, const void* weight, const void* bias,
                        int T, int H, int kind, double eps, int dtype, void* sum, void* y,
                        float* mean, float* rstd, void* stream) {
  const int rc = check(T, H, kind, dtype);
  if (rc != MOE_OK) return rc;
  if (!(eps >= 0.0 && eps <= 3.4e38)) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!x || !weight || !y || (residual && (!sum || sum == y))) return MOE_EINVAL;
  for (const void* q : {x, residual, weight, bias, static_cast<const void*>(sum),
                        static_cast<const void*>(y)})
    if (!aligned16(q)) return MOE_EINVAL;
  const Forward a{x, residual, weight, bias, T, H, kind == MOE_NORM_RMS, static_cast<float>(eps),
                  sum, y, mean, rstd};
  return dtype == MOE_BF16 ? forward<Bf16>(a, dtype, as_stream(stream))
                           : forward<F32>(a, dtype, as_stream(stream));
}

extern "C" size_t moe_norm_backward_workspace_size(int T, int H, int dtype) {
  if (check(T, H, MOE_NORM_LAYER, dtype) != MOE_OK) return 0;
  return static_cast<size_t>(sum_blocks(T, H, dtype)) * 2 * H * 4 + 256;
}

extern "C" int moe_norm_backward(const void* dy, const void* s, const void* weight,
                                 const float* mean, const float* rstd, const void* dsum, int T,
                                 int H, int kind, int dtype, void* dx, void* dweight, void* dbias,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check(T, H, kind, dtype);
  if (rc != MOE_OK) return rc;
  if (T > 0 && ((!dx && !dweight && !dbias) || !dy || !s || !rstd || (dx && !weight) ||
                (kind == MOE_NORM_LAYER && !mean) || !workspace ||
                workspace_bytes < moe_norm_backward_workspace_size(T, H, dtype)))
    return MOE_EINVAL;
  for (const void* q : {dy, s, weight, dsum, static_cast<const void*>(dx),
                        static_cast<const void*>(dweight), static_cast<const void*>(dbias),
                        static_cast<const void*>(workspace)})
    if (!aligned16(q)) return MOE_EINVAL;
  const Backward a{dy, s, weight, kind == MOE_NORM_LAYER ? mean : nullptr, rstd, dsum, T, H, dx,
                   dweight, dbias, nullptr};
  float* ws = static_cast<float*>(workspace);
  return dtype == MOE_BF16 ? backward<Bf16>(a, dtype, ws, as_stream(stream))
                           : backward<F32>(a, dtype, ws, as_stream(stream));
}
