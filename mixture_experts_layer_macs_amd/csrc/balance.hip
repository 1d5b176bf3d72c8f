// moe_balance_loss and moe_router_backward: the router's training losses and
// the gradient of its logits.
//
// With p = softmax(z_t), c_j the slots that name expert j, n the unmasked
// tokens and lse_t = log sum_j exp z_tj,
//   balance = N / (k n) sum_j c_j P_j,   P_j = (1/n) sum_t p_tj
//   z loss  = (1/n) sum_t lse_t^2
//   dz_tj   = p_tj (u_tj - sum_i p_ti u_ti) + dL/dz_loss 2 lse_t p_tj / n,
//   u_tj    = dL/dbalance N c_j / (k n^2) + sum_{s: id_ts = j} dL/dgate_ts
// (the counts carry no gradient).  Both passes read the logits once; a wave
// owns a token, its N logits in registers.
#include <algorithm>
#include <type_traits>

#include "common.h"

namespace moe {
namespace bal {

constexpr int NTHR = 256, WAVES = NTHR / MOE_WAVE;
constexpr int MAX_BLOCKS = 256;

struct Part {  // partial sums of one workgroup, in the workspace
  double* prob;    // [G][N]
  int32_t* count;  // [G][N]
  double* zsq;     // [G]
  int32_t* n;      // [G]
};

__device__ __forceinline__ bool counted(const uint8_t* mask, int t) {
  return mask == nullptr || mask[t] != 0;
}

// Lane l owns experts l, l + 64, ...  A row whose logits are all -inf has no
// probabilities: it counts as a token and adds nothing else.
template <int KPL>
__global__ __launch_bounds__(NTHR) void loss_kernel(const float* __restrict__ logits,
                                                    const int32_t* __restrict__ ids,
                                                    const uint8_t* __restrict__ mask, int T,
                                                    int N, int k, float* __restrict__ lse,
                                                    Part part) {
  __shared__ int32_t s_count[1024];
  __shared__ double s_prob[1024];
  __shared__ double s_z[WAVES];
  __shared__ int32_t s_n[WAVES];
  const int lane = lane_id(), wave = threadIdx.x / MOE_WAVE;
  for (int j = threadIdx.x; j < N; j += NTHR) s_count[j] = 0;
  __syncthreads();
  float pf[KPL];
  double pd[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    pf[i] = 0.f;
    pd[i] = 0.0;
  }
  double zsq = 0.0;
  int n = 0, since = 0;
  for (int t = blockIdx.x * WAVES + wave; t < T; t += gridDim.x * WAVES) {
    if (!counted(mask, t)) {
      if (lane == 0) lse[t] = 0.f;
      continue;
    }
    ++n;
    float z[KPL], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int j = lane + 64 * i;
      z[i] = j < N ? logits[static_cast<size_t>(t) * N + j] : -INFINITY;
      top = fmaxf(top, z[i]);
    }
    for (int s = lane; s < k; s += MOE_WAVE) {
      const int id = ids[static_cast<size_t>(t) * k + s];
      if (static_cast<unsigned>(id) < static_cast<unsigned>(N)) atomicAdd(&s_count[id], 1);
    }
    top = wave_max(top);
    if (top == -INFINITY) {
      if (lane == 0) lse[t] = -INFINITY;
      continue;
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      z[i] = expf(z[i] - top);
      sum += z[i];
    }
    sum = wave_sum(sum);
    const float inv = 1.f / sum, l = top + logf(sum);
#pragma unroll
    for (int i = 0; i < KPL; ++i) pf[i] += z[i] * inv;
    if (lane == 0) lse[t] = l;
    zsq += static_cast<double>(l) * l;
    if (++since == 32) {  // short fp32 runs, long sums in fp64
      since = 0;
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        pd[i] += pf[i];
        pf[i] = 0.f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < KPL; ++i) pd[i] += pf[i];
  if (lane == 0) {
    s_z[wave] = zsq;
    s_n[wave] = n;
  }
  for (int w = 0; w < WAVES; ++w) {  // wave order: the same sum every time
    if (wave == w)
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        const int j = lane + 64 * i;
        if (j < N) s_prob[j] = (w ? s_prob[j] : 0.0) + pd[i];
      }
    __syncthreads();
  }
  const size_t g = blockIdx.x;
  for (int j = threadIdx.x; j < N; j += NTHR) {
    part.prob[g * N + j] = s_prob[j];
    part.count[g * N + j] = s_count[j];
  }
  if (threadIdx.x == 0) {
    double z = 0.0;
    int m = 0;
    for (int w = 0; w < WAVES; ++w) {
      z += s_z[w];
      m += s_n[w];
    }
    part.zsq[g] = z;
    part.n[g] = m;
  }
}

__global__ __launch_bounds__(1024) void finish_kernel(Part part, int G, int N, int k,
                                                      float* __restrict__ losses,
                                                      int32_t* __restrict__ counts,
                                                      float* __restrict__ mean_prob) {
  __shared__ double s_dot[16];
  __shared__ int s_total;
  if (threadIdx.x == 0) {
    int n = 0;
    for (int g = 0; g < G; ++g) n += part.n[g];
    s_total = n;
  }
  __syncthreads();
  const int n = s_total;
  const double inv = n > 0 ? 1.0 / n : 0.0;
  double dot = 0.0;
  const int j = threadIdx.x;
  if (j < N) {
    double p = 0.0;
    int c = 0;
    for (int g = 0; g < G; ++g) {
      p += part.prob[static_cast<size_t>(g) * N + j];
      c += part.count[static_cast<size_t>(g) * N + j];
    }
    p *= inv;
    counts[j] = c;
    mean_prob[j] = static_cast<float>(p);
    dot = p * c;
  }
  dot = wave_sum_f64(dot);
  if (lane_id() == 0) s_dot[threadIdx.x / MOE_WAVE] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    double d = 0.0, z = 0.0;
    for (int w = 0; w < 16; ++w) d += s_dot[w];
    for (int g = 0; g < G; ++g) z += part.zsq[g];
    losses[0] = static_cast<float>(d * inv * N / k);
    losses[1] = static_cast<float>(z * inv);
    counts[N] = n;
  }
}

__device__ __forceinline__ void store_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_elem(__bf16* p, float v) { *p = static_cast<__bf16>(v); }

template <int KPL, typename E>
__global__ __launch_bounds__(NTHR) void grad_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ mask, const float* __restrict__ lse,
    const int32_t* __restrict__ counts, const float* __restrict__ d_losses,
    const float* __restrict__ d_gates, int T, int N, int k, E* __restrict__ dlogits) {
  const int lane = lane_id(), wave = threadIdx.x / MOE_WAVE;
  const double n = counts[N];
  const float db = d_losses ? d_losses[0] : 0.f, dzl = d_losses ? d_losses[1] : 0.f;
  const double inv = n > 0 ? 1.0 / n : 0.0;
  float base[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int j = lane + 64 * i;
    base[i] = j < N ? static_cast<float>(db * inv * inv * N / k * counts[j]) : 0.f;
  }
  const float zc = static_cast<float>(2.0 * dzl * inv);
  for (int t = blockIdx.x * WAVES + wave; t < T; t += gridDim.x * WAVES) {
    const size_t row = static_cast<size_t>(t) * N;
    const float l = lse[t];
    if (!counted(mask, t) || l == -INFINITY) {
#pragma unroll
      for (int i = 0; i < KPL; ++i)
        if (lane + 64 * i < N) store_elem(&dlogits[row + lane + 64 * i], 0.f);
      continue;
    }
    float p[KPL], u[KPL];
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int j = lane + 64 * i;
      p[i] = j < N ? expf(logits[row + j] - l) : 0.f;
      u[i] = base[i];
    }
    if (d_gates) {
      for (int s0 = 0; s0 < k; s0 += MOE_WAVE) {
        const int s = s0 + lane;
        const int id = s < k ? ids[static_cast<size_t>(t) * k + s] : -1;
        const float dg = s < k ? d_gates[static_cast<size_t>(t) * k + s] : 0.f;
        const int m = min(MOE_WAVE, k - s0);
        for (int q = 0; q < m; ++q) {
          const int e = read_lane(id, q);
          const float d = __uint_as_float(read_lane(__float_as_uint(dg), q));
#pragma unroll
          for (int i = 0; i < KPL; ++i) u[i] += e == lane + 64 * i ? d : 0.f;
        }
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) dot += p[i] * u[i];
    dot = wave_sum(dot);
    const float shift = zc * l - dot;
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if (lane + 64 * i < N) store_elem(&dlogits[row + lane + 64 * i], p[i] * (u[i] + shift));
  }
}

inline int blocks(int T) {
  const int b = (T + WAVES - 1) / WAVES;
  return b < 1 ? 1 : b > MAX_BLOCKS ? MAX_BLOCKS : b;
}

inline size_t part_bytes(int G, int N) {
  return static_cast<size_t>(G) * (N + 1) * 12 + 64;
}

template <typename F>
void by_width(int N, F f) {
  if (N <= 64) f(std::integral_constant<int, 1>{});
  else if (N <= 128) f(std::integral_constant<int, 2>{});
  else if (N <= 256) f(std::integral_constant<int, 4>{});
  else if (N <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

}  // namespace bal
}  // namespace moe

using namespace moe;
using namespace moe::bal;

extern "C" size_t moe_balance_workspace_size(int T, int N) {
  if (T < 0 || T > (1 << 20) || N < 1 || N > 1024) return 0;
  return part_bytes(blocks(T), N);
}

extern "C" int moe_balance_loss(const float* logits, const int32_t* slot_ids,
                                const uint8_t* token_mask, int T, int N, int k, float* losses,
                                int32_t* counts, float* mean_prob, float* lse, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (T < 0 || T > (1 << 20) || N < 1 || N > 1024 || k < 1 || k > N) return MOE_EINVAL;
  if (!losses || !counts || !mean_prob || !workspace) return MOE_EINVAL;
  if (T > 0 && (!logits || !slot_ids || !lse)) return MOE_EINVAL;
  const int G = blocks(T);
  if (workspace_bytes < part_bytes(G, N) || reinterpret_cast<uintptr_t>(workspace) % 8 != 0)
    return MOE_EINVAL;
  Part p;
  p.prob = static_cast<double*>(workspace);
  p.zsq = p.prob + static_cast<size_t>(G) * N;
  p.count = reinterpret_cast<int32_t*>(p.zsq + G);
  p.n = p.count + static_cast<size_t>(G) * N;
  hipStream_t s = as_stream(stream);
  by_width(N, [&](auto c) {
    hipLaunchKernelGGL(loss_kernel<decltype(c)::value>, dim3(G), dim3(NTHR), 0, s, logits,
                       slot_ids, token_mask, T, N, k, lse, p);
  });
  hipLaunchKernelGGL(finish_kernel, dim3(1), dim3(1024), 0, s, p, G, N, k, losses, counts,
                     mean_prob);
  return launch_status();
}

extern "C" int moe_router_backward(const float* logits, const int32_t* topk_ids,
                                   const uint8_t* token_mask, const float* lse,
                                   const int32_t* counts, const float* d_losses,
                                   const float* d_gates, int T, int N, int k, int dtype,
                                   void* dlogits, void* stream) {
  if (T < 0 || T > (1 << 20) || N < 1 || N > 1024 || k < 1 || k > N) return MOE_EINVAL;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EUNSUP;
  if (T == 0) return MOE_OK;
  if (!logits || !lse || !counts || !dlogits || (d_gates && !topk_ids)) return MOE_EINVAL;
  hipStream_t s = as_stream(stream);
  const int G = std::min((T + WAVES - 1) / WAVES, cu_count() * 8);
  by_width(N, [&](auto c) {
    constexpr int KPL = decltype(c)::value;
    if (dtype == MOE_F32)
      hipLaunchKernelGGL((grad_kernel<KPL, float>), dim3(G), dim3(NTHR), 0, s, logits, topk_ids,
                         token_mask, lse, counts, d_losses, d_gates, T, N, k,
                         static_cast<float*>(dlogits));
    else
      hipLaunchKernelGGL((grad_kernel<KPL, __bf16>), dim3(G), dim3(NTHR), 0, s, logits, topk_ids,
                         token_mask, lse, counts, d_losses, d_gates, T, N, k,
                         static_cast<__bf16*>(dlogits));
  });
  return launch_status();
}
