// Activations and the output epilogue of the dense layer.
#pragma once

#include "common.h"

namespace moe {
namespace lin {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------- element types: vectors
struct Bf16 {
  typedef uint16_t elem;
  static constexpr int V = 8;  // elements in 16 bytes
};
struct F32 {
  typedef float elem;
  static constexpr int V = 4;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {  // round to nearest even
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ void load4(const uint16_t* p, float* f) {
  const u32x2 w = *reinterpret_cast<const u32x2*>(p);
  f[0] = __uint_as_float(w.x << 16);
  f[1] = __uint_as_float(w.x & 0xffff0000u);
  f[2] = __uint_as_float(w.y << 16);
  f[3] = __uint_as_float(w.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const float* p, float* f) {
  const f32x4 v = *reinterpret_cast<const f32x4*>(p);
  f[0] = v.x;
  f[1] = v.y;
  f[2] = v.z;
  f[3] = v.w;
}
__device__ __forceinline__ void store4(uint16_t* p, const float* f) {
  *reinterpret_cast<u32x2*>(p) = u32x2{pack2(f[0], f[1]), pack2(f[2], f[3])};
}
__device__ __forceinline__ void store4(float* p, const float* f) {
  *reinterpret_cast<f32x4*>(p) = f32x4{f[0], f[1], f[2], f[3]};
}
// V values, 4 or (16 bytes of bf16) 8
template <int V>
__device__ __forceinline__ void load_v(const uint16_t* p, float* f) {
  if constexpr (V == 8) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    load4(p, f);
  }
}
template <int V>
__device__ __forceinline__ void load_v(const float* p, float* f) {
#pragma unroll
  for (int i = 0; i < V; i += 4) load4(p + i, f + i);
}
template <int V>
__device__ __forceinline__ void store_v(uint16_t* p, const float* f) {
  if constexpr (V == 8)
    *reinterpret_cast<u32x4*>(p) = u32x4{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]),
                                         pack2(f[6], f[7])};
  else
    store4(p, f);
}
template <int V>
__device__ __forceinline__ void store_v(float* p, const float* f) {
#pragma unroll
  for (int i = 0; i < V; i += 4) store4(p + i, f + i);
}
__device__ __forceinline__ void store1(uint16_t* p, float v) {
  *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// ------------------------------------------------------------- activations
// The hardware exponential and reciprocal (about one unit each); the rounded
// argument of the exponential costs |a| 2^-24 relative.
__device__ __forceinline__ float sigmoid(float a) {
  return __builtin_amdgcn_rcpf(1.f + __expf(-a));
}

// Outside +-SILU_END sigmoid is 0 or 1 in fp32.  Its factor a is held there
// where an infinite one would give inf * 0 for a limit of 0; NaN stays.
constexpr float SILU_END = 128.f;

// silu(a) and silu'(a), s = sigmoid(a)
__device__ __forceinline__ float silu(float a, float s) {
  return (a < -SILU_END ? -SILU_END : a) * s;
}
__device__ __forceinline__ float silu_slope(float a, float s) {
  const float z = a < -SILU_END ? -SILU_END : a > SILU_END ? SILU_END : a;
  return s * (1.f + z * (1.f - s));
}

// Phi(-m) of the normal distribution for m >= 0 and, in *density, exp(-m^2/2):
//   Phi(-m) = exp(-m^2/2) t Q(t),  t = 1 / (1 + c m),
// Q a least-maximum fit of the relative error on 0 <= m <= 13.5, where fp32's
// range ends.  bf16 results take 7 coefficients (8e-7, 7 units of fp32 where the
// tail is 1/2: the bias gradient sums unrounded slopes), fp32 ones 9 (5e-8; the
// exponential's rounded argument adds m^2 2^-23).  The tail is relative to
// itself, not to 1, so that gelu of -4 is as exact as that of 4; it shares its
// exponential with the density.  These instructions are what a wide layer's
// epilogue costs: about 30 us of 450 for a 4096 x 14336 output.
template <typename E>
__device__ __forceinline__ float normal_tail(float m, float* density) {
  constexpr bool WIDE = sizeof(E) == 4;
  const float t = __builtin_amdgcn_rcpf(1.f + (WIDE ? 0.25f : 0.36f) * m);
  const float e = __builtin_amdgcn_exp2f(m * m * -0.72134752f);  // -1 / (2 ln 2)
  float p;
  if constexpr (WIDE) {
    p = 0.0262954589f;
    p = p * t - 0.155636474f;
    p = p * t + 0.30207628f;
    p = p * t - 0.212748349f;
    p = p * t + 0.206696898f;
    p = p * t + 0.030758867f;
    p = p * t + 0.104321837f;
    p = p * t + 0.0984327942f;
    p = p * t + 0.099802658f;
  } else {
    p = 0.0473445766f;
    p = p * t - 0.180751696f;
    p = p * t + 0.182297647f;
    p = p * t + 0.025623776f;
    p = p * t + 0.140057445f;
    p = p * t + 0.141710669f;
    p = p * t + 0.143717438f;
  }
  *density = e;
  return p * t * e;
}

constexpr float TAIL_END = 16.f;  // exp(-m^2/2) is 0 in fp32 from 14 on

__device__ __forceinline__ float relu(float z) { return z < 0.f ? 0.f : z; }  // NaN stays

// E: the type that the result is rounded to
template <typename E>
__device__ __forceinline__ float act_value(int act, float z) {
  float e;
  switch (act) {
    case MOE_ACT_RELU: return relu(z);
    case MOE_ACT_SILU: return silu(z, sigmoid(z));
    case MOE_ACT_GELU: {  // z Phi(z) = max(z, 0) - |z| Phi(-|z|)
      const float m = fminf(fabsf(z), TAIL_END);
      return relu(z) - m * normal_tail<E>(m, &e);
    }
    default: return z;
  }
}

template <typename E>
__device__ __forceinline__ float act_slope(int act, float z) {
  switch (act) {
    case MOE_ACT_SILU: return silu_slope(z, sigmoid(z));
    case MOE_ACT_GELU: {  // Phi(z) + z phi(z)
      const float m = fabsf(z) > TAIL_END ? TAIL_END : fabsf(z);  // NaN stays
      float e;
      const float tail = normal_tail<E>(m, &e), rise = m * 0.39894228040143268f * e;
      return z < 0.f ? tail - rise : 1.f - tail + rise;
    }
    default: return 1.f;
  }
}

// ------------------------------------------------------------------ output
// What follows the product: bias, z, activation, residual, y.
struct Epilogue {
  const void *bias, *residual;
  void *z, *y;
  int act;
};

// Columns n .. n + V - 1 of row m; N: columns of y.  GLU: g and u are the gate
// and up sums of those columns.  residual may be y: each element is read by
// the lane that writes it, before it does.
template <typename E, bool GLU, int V>
__device__ __forceinline__ void finish(const Epilogue& e, int m, int n, int N, float* g, float* u) {
  const size_t at = static_cast<size_t>(m) * N + n;
  float r[V];
  if (e.residual) load_v<V>(static_cast<const E*>(e.residual) + at, r);
  if (e.bias) {
    float b[V];
    load_v<V>(static_cast<const E*>(e.bias) + n, b);
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] += b[i];
    if constexpr (GLU) {
      load_v<V>(static_cast<const E*>(e.bias) + N + n, b);
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] += b[i];
    }
  }
  if (e.z) {
    E* z = static_cast<E*>(e.z) + (GLU ? at + static_cast<size_t>(m) * N : at);
    store_v<V>(z, g);
    if constexpr (GLU) store_v<V>(z + N, u);
  }
  float v[V];
  if constexpr (GLU) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = silu(g[i], sigmoid(g[i])) * u[i];
  } else {
    if (e.act == MOE_ACT_GELU) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = act_value<E>(MOE_ACT_GELU, g[i]);
    } else if (e.act == MOE_ACT_SILU) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = act_value<E>(MOE_ACT_SILU, g[i]);
    } else if (e.act == MOE_ACT_RELU) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = act_value<E>(MOE_ACT_RELU, g[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = g[i];
    }
  }
  if (e.residual) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += r[i];
  }
  store_v<V>(static_cast<E*>(e.y) + at, v);
}

// ----------------------------------------------------------- bias gradient
// Column sums of [blocks][W] partial sums, 64 columns per workgroup of 256
// threads; red: 256 floats of LDS.
struct BiasSum {
  const float* part;
  int blocks, W;
  void* dbias;
};

template <typename E>
__device__ __forceinline__ void bias_sum(const BiasSum& b, int block, float* red) {
  const int c = threadIdx.x % 64, r = threadIdx.x / 64, o = block * 64 + c;
  float v = 0.f;
  if (o < b.W)
#pragma unroll 8
    for (int i = r; i < b.blocks; i += 4) v += b.part[static_cast<size_t>(i) * b.W + o];
  red[threadIdx.x] = v;
  __syncthreads();
  if (r == 0 && o < b.W)
    store1(static_cast<E*>(b.dbias) + o, (red[c] + red[64 + c]) + (red[128 + c] + red[192 + c]));
}

}  // namespace lin
}  // namespace moe
