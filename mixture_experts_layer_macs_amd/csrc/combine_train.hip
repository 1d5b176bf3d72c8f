// moe_combine_dropout and moe_combine_backward: the gate-weighted combine
// ("MACS", §3.1 Eq. 1) of a training step,
//   y[t]           = residual[t] + m[t] * sum_{s kept} g[t,s] out_rows[row(t,s)]
//   d_out_rows[r]  = g[t,s] (m[t] * dy[t]),   r = row(t,s)
//   d_gates[t,s]   = < out_rows[r], m[t] * dy[t] >
// where m is the dropout factor of each element, 0 or 1/(1-p).  The factor is
// computed from the element's position where it is needed and never stored:
// word e % 4 of Philox4x32-10 (J. Salmon et al., "Parallel random numbers: as
// easy as 1, 2, 3", 2011) with the seed as key and (e / 4, offset) as counter
// decides element e = t H + c, which is kept if the word is at least
// floor(p 2^32).
//
// Both passes are bound by HBM: the k expert rows of a token are read (and in
// the backward pass written) once.  A power-of-two group of threads owns a
// token, 16 bytes of a row per thread and step, up to 8 rows in flight; the
// mask's integer work runs while they are.
//
// Measured, 8192 tokens of 8 rows of 2048 bf16, p = 0.1: forward with residual
// 63 us (322 MB, 5.1 TB/s; a plain read of 268 MB takes 59), the same without
// dropout; backward 111 us (543 MB, 4.9 TB/s; a large copy runs at 4.8).
#include "common.h"

namespace moe {
namespace ctr {

constexpr int NTHR = 256;
constexpr int SB = 8;  // slots in flight per thread

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// 16 bytes of a row: 8 bf16 or 4 fp32 values.
struct Bf16 {
  static constexpr int V = 8;
  typedef uint16_t elem;
  static __device__ __forceinline__ void unpack(uint4 q, float* f) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // round to nearest even
      const f32x2 v = {f[2 * i], f[2 * i + 1]};
      w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
struct F32 {
  static constexpr int V = 4;
  typedef float elem;
  static __device__ __forceinline__ void unpack(uint4 q, float* f) {
    f[0] = __uint_as_float(q.x);
    f[1] = __uint_as_float(q.y);
    f[2] = __uint_as_float(q.z);
    f[3] = __uint_as_float(q.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

struct Drop {
  const uint64_t* rng;  // {seed, offset}, read on the device; null without dropout
  uint32_t threshold;
  float scale;
};

// Bit i: element e + i is kept, for V elements from e (a multiple of 4).
template <int V>
__device__ __forceinline__ uint32_t keep_bits(uint64_t e, uint64_t seed, uint64_t offset,
                                              uint32_t threshold) {
  uint32_t bits = 0;
#pragma unroll
  for (int b = 0; b < V / 4; ++b) {
    const uint64_t ctr = e / 4 + b;
    uint32_t c0 = static_cast<uint32_t>(ctr), c1 = static_cast<uint32_t>(ctr >> 32);
    uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
    uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      // one 64-bit multiply-add gives both halves of a product
      const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0;
      const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
      c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
      c1 = static_cast<uint32_t>(p1);
      c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
      c3 = static_cast<uint32_t>(p0);
      k0 += 0x9E3779B9u;
      k1 += 0xBB67AE85u;
    }
    const uint32_t w[4] = {c0, c1, c2, c3};
#pragma unroll
    for (int i = 0; i < 4; ++i) bits |= w[i] >= threshold ? 1u << (4 * b + i) : 0u;
  }
  return bits;
}

// f *= m; a dropped element becomes 0 whatever it held.
template <int V>
__device__ __forceinline__ void apply_mask(float* f, uint32_t bits, float scale) {
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = bits >> i & 1 ? f[i] * scale : 0.f;
}

template <typename D>
__global__ __launch_bounds__(NTHR) void forward_kernel(
    const typename D::elem* __restrict__ rows, const int32_t* __restrict__ slot_row,
    const float* __restrict__ gates, const typename D::elem* residual, Drop drop, int T, int k,
    int H, int tpt, typename D::elem* y) {
  constexpr int V = D::V;
  const int t = blockIdx.x * (NTHR / tpt) + threadIdx.x / tpt;
  if (t >= T) return;
  const int nv = H / V;
  uint64_t seed = 0, offset = 0;
  if (drop.rng) {
    seed = drop.rng[0];
    offset = drop.rng[1];
  }
  for (int v = threadIdx.x % tpt; v < nv; v += tpt) {
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    const size_t e = static_cast<size_t>(t) * H + v * V;
    uint4 rq = make_uint4(0, 0, 0, 0);
    uint32_t keep = 0;
    for (int s0 = 0; s0 < k; s0 += SB) {
      int r[SB];
      float g[SB];
      uint4 q[SB];
#pragma unroll
      for (int u = 0; u < SB; ++u) {
        const bool in = s0 + u < k;
        const size_t at = static_cast<size_t>(t) * k + s0 + u;
        r[u] = in ? slot_row[at] : -1;
        g[u] = in ? gates[at] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < SB; ++u)
        if (r[u] >= 0)
          q[u] = *reinterpret_cast<const uint4*>(rows + static_cast<size_t>(r[u]) * H + v * V);
      if (s0 == 0) {  // the mask is computed while the first rows are in flight
        if (residual) rq = *reinterpret_cast<const uint4*>(residual + e);
        if (drop.rng) keep = keep_bits<V>(e, seed, offset, drop.threshold);
      }
#pragma unroll
      for (int u = 0; u < SB; ++u) {
        if (r[u] < 0) continue;
        float f[V];
        D::unpack(q[u], f);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += g[u] * f[i];
      }
    }
    if (drop.rng) apply_mask<V>(acc, keep, drop.scale);
    if (residual) {
      float f[V];
      D::unpack(rq, f);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += f[i];
    }
    *reinterpret_cast<uint4*>(y + e) = D::pack(acc);
  }
}

// Sum of v over the threads of a token (tpt, a power of two) in this wave.
__device__ __forceinline__ float wave_part(float v, int tpt) {
  for (int m = 1; m < tpt && m < MOE_WAVE; m *= 2) v += __shfl_xor(v, m, MOE_WAVE);
  return v;
}

template <typename D>
__global__ __launch_bounds__(NTHR) void backward_kernel(
    const typename D::elem* __restrict__ dy, const typename D::elem* __restrict__ rows,
    const int32_t* __restrict__ slot_row, const float* __restrict__ gates, Drop drop, int T,
    int k, int H, int tpt, typename D::elem* __restrict__ d_rows, float* __restrict__ d_gates) {
  constexpr int V = D::V;
  __shared__ float red[NTHR / MOE_WAVE][SB];
  const int t = blockIdx.x * (NTHR / tpt) + threadIdx.x / tpt;
  const bool live = t < T;
  const int nv = live ? H / V : 0;
  uint64_t seed = 0, offset = 0;
  if (drop.rng) {
    seed = drop.rng[0];
    offset = drop.rng[1];
  }
  for (int s0 = 0; s0 < k; s0 += SB) {
    int r[SB];
    float g[SB], dot[SB];
#pragma unroll
    for (int u = 0; u < SB; ++u) {
      const bool in = live && s0 + u < k;
      const size_t at = static_cast<size_t>(t) * k + s0 + u;
      r[u] = in ? slot_row[at] : -1;
      g[u] = in ? gates[at] : 0.f;
      dot[u] = 0.f;
    }
    for (int v = threadIdx.x % tpt; v < nv; v += tpt) {
      uint4 q[SB];
      if (d_gates) {
#pragma unroll
        for (int u = 0; u < SB; ++u)
          if (r[u] >= 0)
            q[u] = *reinterpret_cast<const uint4*>(rows + static_cast<size_t>(r[u]) * H + v * V);
      }
      const size_t e = static_cast<size_t>(t) * H + v * V;
      float d[V];
      D::unpack(*reinterpret_cast<const uint4*>(dy + e), d);
      if (drop.rng)
        apply_mask<V>(d, keep_bits<V>(e, seed, offset, drop.threshold), drop.scale);
#pragma unroll
      for (int u = 0; u < SB; ++u) {
        if (r[u] < 0) continue;
        if (d_gates) {
          float f[V];
          D::unpack(q[u], f);
#pragma unroll
          for (int i = 0; i < V; ++i) dot[u] += f[i] * d[i];
        }
        if (d_rows) {
          float f[V];
#pragma unroll
          for (int i = 0; i < V; ++i) f[i] = g[u] * d[i];
          *reinterpret_cast<uint4*>(d_rows + static_cast<size_t>(r[u]) * H + v * V) = D::pack(f);
        }
      }
    }
    if (!d_gates) continue;
#pragma unroll
    for (int u = 0; u < SB; ++u) dot[u] = wave_part(dot[u], tpt);
    if (tpt > MOE_WAVE) {
      __syncthreads();
      if (lane_id() == 0)
#pragma unroll
        for (int u = 0; u < SB; ++u) red[threadIdx.x / MOE_WAVE][u] = dot[u];
      __syncthreads();
      const int w0 = threadIdx.x / tpt * (tpt / MOE_WAVE);
#pragma unroll
      for (int u = 0; u < SB; ++u) {
        dot[u] = 0.f;
        for (int w = 0; w < tpt / MOE_WAVE; ++w) dot[u] += red[w0 + w][u];
      }
    }
    if (live && threadIdx.x % tpt == 0)
#pragma unroll
      for (int u = 0; u < SB; ++u)
        if (s0 + u < k) d_gates[static_cast<size_t>(t) * k + s0 + u] = dot[u];
  }
}

// Threads of a token: the smallest power of two that covers a row in one
// step, at most a workgroup.
inline int threads_per_token(int H, int V) {
  int n = 1;
  while (n < NTHR && n * V < H) n *= 2;
  return n;
}

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

inline int check(int T, int k, int H, int dtype, double p, const uint64_t* rng, Drop* drop) {
  if (T < 0 || T > (1 << 20) || k < 1 || k > 1024 || H < 1 || !(p >= 0.0 && p < 1.0))
    return MOE_EINVAL;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EUNSUP;
  if (H % 8 != 0) return MOE_EUNSUP;
  if (T > 0 && p > 0.0 && (!rng || reinterpret_cast<uintptr_t>(rng) % 8 != 0)) return MOE_EINVAL;
  drop->rng = p > 0.0 ? rng : nullptr;
  drop->threshold = static_cast<uint32_t>(p * 4294967296.0);
  drop->scale = static_cast<float>(1.0 / (1.0 - p));
  return MOE_OK;
}

}  // namespace ctr
}  // namespace moe

using namespace moe;
using namespace moe::ctr;

extern "C" int moe_combine_dropout(const void* out_rows, const int32_t* slot_row,
                                   const float* topk_gates, const void* residual, double p,
                                   const uint64_t* rng, int T, int k, int H, int dtype, void* y,
                                   void* stream) {
  Drop drop;
  const int rc = check(T, k, H, dtype, p, rng, &drop);
  if (rc != MOE_OK || T == 0) return rc;
  if (!out_rows || !slot_row || !topk_gates || !y) return MOE_EINVAL;
  if (!aligned16(out_rows) || !aligned16(residual) || !aligned16(y)) return MOE_EINVAL;
  hipStream_t s = as_stream(stream);
  auto go = [&](auto d) {
    using D = decltype(d);
    typedef typename D::elem E;
    const int tpt = threads_per_token(H, D::V), per = NTHR / tpt;
    hipLaunchKernelGGL(forward_kernel<D>, dim3((T + per - 1) / per), dim3(NTHR), 0, s,
                       static_cast<const E*>(out_rows), slot_row, topk_gates,
                       static_cast<const E*>(residual), drop, T, k, H, tpt, static_cast<E*>(y));
  };
  if (dtype == MOE_BF16) go(Bf16{});
  else go(F32{});
  return launch_status();
}

extern "C" int moe_combine_backward(const void* dy, const void* out_rows,
                                    const int32_t* slot_row, const float* topk_gates, double p,
                                    const uint64_t* rng, int T, int k, int H, int dtype,
                                    void* d_out_rows, float* d_gates, void* stream) {
  Drop drop;
  const int rc = check(T, k, H, dtype, p, rng, &drop);
  if (rc != MOE_OK || T == 0) return rc;  // empty outputs may have null addresses
  if (!d_out_rows && !d_gates) return MOE_EINVAL;
  if (!dy || !slot_row || !topk_gates || (d_gates && !out_rows)) return MOE_EINVAL;
  if (!aligned16(dy) || !aligned16(out_rows) || !aligned16(d_out_rows)) return MOE_EINVAL;
  hipStream_t s = as_stream(stream);
  auto go = [&](auto d) {
    using D = decltype(d);
    typedef typename D::elem E;
    const int tpt = threads_per_token(H, D::V), per = NTHR / tpt;
    hipLaunchKernelGGL(backward_kernel<D>, dim3((T + per - 1) / per), dim3(NTHR), 0, s,
                       static_cast<const E*>(dy), static_cast<const E*>(out_rows), slot_row,
                       topk_gates, drop, T, k, H, tpt, static_cast<E*>(d_out_rows), d_gates);
  };
  if (dtype == MOE_BF16) go(Bf16{});
  else go(F32{});
  return launch_status();
}
