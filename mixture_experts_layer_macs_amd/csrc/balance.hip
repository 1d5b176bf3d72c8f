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

constexpr int NTHR = 1024, WAVES = NTHR / MOE_WAVE;
constexpr int COLS = 256;  // columns of the cross-wave sums held in LDS at once

// GL lanes own a token (the smallest power of two from 8 to 64 that covers N),
// lane l of them experts l, l + GL, ...: a wave takes 64 / GL tokens at once,
// so a router of few experts does not leave lanes idle.
template <typename T, int GL, class Op>
__device__ __forceinline__ T group_reduce(T v, Op op) {
  v = op(v, dpp_t<T, DPP_QUAD_1032>(v, v));
  v = op(v, dpp_t<T, DPP_QUAD_2301>(v, v));
  v = op(v, dpp_t<T, DPP_ROW_HALF_MIRROR>(v, v));
  if constexpr (GL > 8) v = op(v, dpp_t<T, 0x140>(v, v));  // lane 15-i of each row
  if constexpr (GL > 16) v = op(v, __shfl_xor(v, 16, MOE_WAVE));
  if constexpr (GL > 32) v = op(v, __shfl_xor(v, 32, MOE_WAVE));
  return v;
}
template <int GL>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<float, GL>(v, [](float a, float b) { return a + b; });
}
template <int GL>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<float, GL>(v, [](float a, float b) { return fmaxf(a, b); });
}

// Partial sums of one workgroup, in the workspace.
struct Part {
  double* zsq;     // [G]
  int32_t* n;      // [G]
  float* prob;     // [G][N]
  int32_t* count;  // [G][N]
  float *losses, *mean_prob;
  int32_t* counts;
  int G, N, k;
};

// The workgroups' sums to the outputs: a thread owns a column in every R-th
// partial row, 8 rows in flight.
__device__ __forceinline__ void finish(const Part& p) {
  __shared__ double s_p[NTHR];
  __shared__ int s_c[NTHR];
  __shared__ double s_dot[WAVES], s_z;
  __shared__ int s_n;
  const int tid = threadIdx.x;
  if (tid < MOE_WAVE) {
    int n = 0;
    double z = 0.0;
    for (int g = tid; g < p.G; g += MOE_WAVE) {
      n += p.n[g];
      z += p.zsq[g];
    }
    n = wave_sum(n);
    z = wave_sum_f64(z);
    if (tid == 0) {
      s_n = n;
      s_z = z;
    }
  }
  int cols = 32;  // threads along the columns: a power of two that covers N
  while (cols < p.N) cols *= 2;
  const int R = NTHR / cols, c = tid & (cols - 1), r = tid / cols;
  double sum = 0.0;
  int count = 0;
  if (c < p.N) {
    for (int g0 = r; g0 < p.G; g0 += 8 * R) {
      float f[8];
      int m[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int g = g0 + u * R;
        f[u] = g < p.G ? p.prob[static_cast<size_t>(g) * p.N + c] : 0.f;
        m[u] = g < p.G ? p.count[static_cast<size_t>(g) * p.N + c] : 0;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        sum += f[u];
        count += m[u];
      }
    }
  }
  s_p[tid] = sum;
  s_c[tid] = count;
  __syncthreads();
  const int n = s_n;
  const double inv = n > 0 ? 1.0 / n : 0.0;
  double dot = 0.0;
  if (tid < p.N) {
    sum = 0.0;
    count = 0;
    for (int i = 0; i < R; ++i) {  // the same order every time
      sum += s_p[i * cols + tid];
      count += s_c[i * cols + tid];
    }
    sum *= inv;
    p.counts[tid] = count;
    p.mean_prob[tid] = static_cast<float>(sum);
    dot = sum * count;
  }
  dot = wave_sum_f64(dot);
  if (lane_id() == 0) s_dot[tid / MOE_WAVE] = dot;
  __syncthreads();
  if (tid == 0) {
    double d = 0.0;
    for (int w = 0; w < WAVES; ++w) d += s_dot[w];
    p.losses[0] = static_cast<float>(d * inv * p.N / p.k);
    p.losses[1] = static_cast<float>(s_z * inv);
    p.counts[p.N] = n;
  }
}

__global__ __launch_bounds__(NTHR) void finish_kernel(Part p) { finish(p); }

// A row whose logits are all -inf has no probabilities: it counts as a token
// and adds nothing else.  The next token's logits are requested before the
// current one is worked on.
template <int GL, int KPL>
__global__ __launch_bounds__(NTHR) void loss_kernel(const float* __restrict__ logits,
                                                    const int32_t* __restrict__ ids,
                                                    const uint8_t* __restrict__ mask, int T,
                                                    float* __restrict__ lse, Part part) {
  constexpr int TPW = MOE_WAVE / GL;
  const int N = part.N, k = part.k;
  __shared__ int32_t s_count[1024];
  __shared__ double s_prob[WAVES][COLS];
  __shared__ double s_z[WAVES];
  __shared__ int32_t s_n[WAVES];
  const int lane = lane_id(), wave = threadIdx.x / MOE_WAVE, gl = lane & (GL - 1);
  for (int j = threadIdx.x; j < N; j += NTHR) s_count[j] = 0;
  __syncthreads();
  float pf[KPL], znext[KPL];
  double pd[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    pf[i] = 0.f;
    pd[i] = 0.0;
  }
  double zsq = 0.0;
  int n = 0, since = 0, idnext = -1;
  bool onnext = false;
  const int step = gridDim.x * WAVES * TPW;
  auto request = [&](int t) {
    const bool in = t < T;
    onnext = in && (mask == nullptr || mask[t] != 0);
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int j = gl + GL * i;
      znext[i] = in && j < N ? logits[static_cast<size_t>(t) * N + j] : -INFINITY;
    }
    idnext = in && gl < k ? ids[static_cast<size_t>(t) * k + gl] : -1;
  };
  const int t0 = (blockIdx.x * WAVES + wave) * TPW;
  request(t0 + lane / GL);
  for (int tb = t0; tb < T; tb += step) {
    const int t = tb + lane / GL;
    float z[KPL], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < KPL; ++i) z[i] = znext[i];
    int id = idnext;
    const bool on = onnext;
    request(t + step);
#pragma unroll
    for (int i = 0; i < KPL; ++i) top = fmaxf(top, z[i]);
    if (on) {
      for (int s = gl; s < k; s += GL) {
        if (s >= GL) id = ids[static_cast<size_t>(t) * k + s];
        if (static_cast<unsigned>(id) < static_cast<unsigned>(N)) atomicAdd(&s_count[id], 1);
      }
    }
    top = group_max<GL>(top);
    const bool some = on && top != -INFINITY;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      z[i] = __expf(z[i] - top);
      sum += z[i];
    }
    sum = group_sum<GL>(sum);
    const float inv = 1.f / sum, l = top + __logf(sum);
#pragma unroll
    for (int i = 0; i < KPL; ++i) pf[i] += some ? z[i] * inv : 0.f;  // padding may hold NaN
    if (gl == 0 && t < T) {
      lse[t] = some ? l : on ? -INFINITY : 0.f;
      n += on;
      if (some) zsq += static_cast<double>(l) * l;
    }
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
  for (int i = 0; i < KPL; ++i) {
    pd[i] += pf[i];
    for (int m = GL; m < MOE_WAVE; m *= 2) pd[i] += __shfl_xor(pd[i], m, MOE_WAVE);
  }
  zsq = wave_sum_f64(zsq);
  n = wave_sum(n);
  if (lane == 0) {
    s_z[wave] = zsq;
    s_n[wave] = n;
  }
  const size_t g = blockIdx.x;
  constexpr int PER = COLS / GL;  // registers of a wave per round
#pragma unroll
  for (int i0 = 0; i0 < KPL; i0 += PER) {
    __syncthreads();
#pragma unroll
    for (int i = i0; i < i0 + PER && i < KPL; ++i)
      if (lane < GL) s_prob[wave][(i - i0) * GL + gl] = pd[i];
    __syncthreads();
    const int j = i0 * GL + threadIdx.x;
    if (threadIdx.x < COLS && j < N && threadIdx.x < (KPL - i0) * GL) {
      double v = 0.0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) v += s_prob[w][threadIdx.x];
      part.prob[g * N + j] = static_cast<float>(v);
      part.count[g * N + j] = s_count[j];
    }
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
  if (gridDim.x == 1) {  // a short batch: one workgroup, one launch
    __syncthreads();
    finish(part);
  }
}

__device__ __forceinline__ void store_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_elem(__bf16* p, float v) { *p = static_cast<__bf16>(v); }

constexpr int GNTHR = 256, GWAVES = GNTHR / MOE_WAVE;

// With GL == 64 the token's slots are the same for the whole wave: ids and
// gate gradients come through scalar registers, and a slot touches the one
// register that holds its expert.  (Comparing every slot with every register
// made this kernel VALU bound: 38 us at 65521 x 256 against 28 us of traffic.)
template <int GL, int KPL, typename E>
__global__ __launch_bounds__(GNTHR) void grad_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ mask, const float* __restrict__ lse,
    const int32_t* __restrict__ counts, const float* __restrict__ d_losses,
    const float* __restrict__ d_gates, int T, int N, int k, E* __restrict__ dlogits) {
  constexpr int TPW = MOE_WAVE / GL;
  const int lane = lane_id(), gl = lane & (GL - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
  const double n = counts[N];
  const float db = d_losses ? d_losses[0] : 0.f, dzl = d_losses ? d_losses[1] : 0.f;
  const double inv = n > 0 ? 1.0 / n : 0.0;
  float base[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int j = gl + GL * i;
    base[i] = j < N ? static_cast<float>(db * inv * inv * N / k * counts[j]) : 0.f;
  }
  const float zc = static_cast<float>(2.0 * dzl * inv);
  const int step = gridDim.x * GWAVES * TPW, t0 = (blockIdx.x * GWAVES + wave) * TPW;
  float znext[KPL], lnext = 0.f;
  bool onnext = false;
  auto request = [&](int t) {
    const bool in = t < T;
    onnext = in && (mask == nullptr || mask[t] != 0);
    lnext = in ? lse[t] : 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int j = gl + GL * i;
      znext[i] = in && j < N ? logits[static_cast<size_t>(t) * N + j] : 0.f;
    }
  };
  request(t0 + lane / GL);
  for (int tb = t0; tb < T; tb += step) {
    const int t = tb + lane / GL;
    const float l = lnext;
    const bool on = onnext && l != -INFINITY;
    float p[KPL], u[KPL];
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      p[i] = gl + GL * i < N ? __expf(znext[i] - l) : 0.f;
      u[i] = base[i];
    }
    request(t + step);
    if (d_gates) {
      if constexpr (GL == MOE_WAVE) {
        const int32_t* idp = ids + static_cast<size_t>(tb) * k;
        const float* dgp = d_gates + static_cast<size_t>(tb) * k;
        for (int q = 0; q < k; ++q) {
          const int e = idp[q], r = e >> 6;
          if (static_cast<unsigned>(e) >= static_cast<unsigned>(N)) continue;
          const float d = lane == (e & 63) ? dgp[q] : 0.f;
          if constexpr (KPL == 1) {
            u[0] += r == 0 ? d : 0.f;
          } else {
#pragma unroll
            for (int i = 0; i < KPL; ++i)
              if (r == i) u[i] += d;
          }
        }
      } else if (t < T) {
        for (int q = 0; q < k; ++q) {
          const int e = ids[static_cast<size_t>(t) * k + q];
          u[0] += e == gl && e < N ? d_gates[static_cast<size_t>(t) * k + q] : 0.f;
        }
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) dot += p[i] * u[i];
    const float shift = zc * l - group_sum<GL>(dot);
    if (t < T) {
#pragma unroll
      for (int i = 0; i < KPL; ++i)
        if (gl + GL * i < N)
          store_elem(&dlogits[static_cast<size_t>(t) * N + gl + GL * i],
                     on ? p[i] * (u[i] + shift) : 0.f);
    }
  }
}

template <typename F>
void by_width(int N, F f) {
  using std::integral_constant;
  if (N <= 8) f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  else if (N <= 16) f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (N <= 32) f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  else if (N <= 64) f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (N <= 128) f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (N <= 256) f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
  else if (N <= 512) f(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  else f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

inline int tokens_per_wave(int N) { return N <= 8 ? 8 : N <= 16 ? 4 : N <= 32 ? 2 : 1; }

// Workgroups of the loss pass: one while a wave has at most 8 rounds, then as
// many as give every wave 4 rounds, at most 256 (the second launch reads
// their sums with one workgroup).
inline int blocks(int T, int N) {
  const int tpb = WAVES * tokens_per_wave(N);  // tokens per round
  if (T <= 8 * tpb) return 1;
  return std::min(256, (T + 4 * tpb - 1) / (4 * tpb));
}

inline size_t part_bytes(int G, int N) { return static_cast<size_t>(G) * (N * 8 + 12) + 64; }

}  // namespace bal
}  // namespace moe

using namespace moe;
using namespace moe::bal;

extern "C" size_t moe_balance_workspace_size(int T, int N) {
  if (T < 0 || T > (1 << 20) || N < 1 || N > 1024) return 0;
  return part_bytes(blocks(T, N), N);
}

extern "C" int moe_balance_loss(const float* logits, const int32_t* slot_ids,
                                const uint8_t* token_mask, int T, int N, int k, float* losses,
                                int32_t* counts, float* mean_prob, float* lse, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (T < 0 || T > (1 << 20) || N < 1 || N > 1024 || k < 1 || k > N) return MOE_EINVAL;
  if (!losses || !counts || !mean_prob || !workspace) return MOE_EINVAL;
  if (T > 0 && (!logits || !slot_ids || !lse)) return MOE_EINVAL;
  const int G = blocks(T, N);
  if (workspace_bytes < part_bytes(G, N) || reinterpret_cast<uintptr_t>(workspace) % 8 != 0)
    return MOE_EINVAL;
  Part p;
  p.zsq = static_cast<double*>(workspace);
  p.n = reinterpret_cast<int32_t*>(p.zsq + G);
  p.count = p.n + G;
  p.prob = reinterpret_cast<float*>(p.count + static_cast<size_t>(G) * N);
  p.losses = losses;
  p.counts = counts;
  p.mean_prob = mean_prob;
  p.G = G;
  p.N = N;
  p.k = k;
  hipStream_t s = as_stream(stream);
  by_width(N, [&](auto gl, auto kpl) {
    hipLaunchKernelGGL((loss_kernel<decltype(gl)::value, decltype(kpl)::value>), dim3(G), dim3(NTHR),
                       0, s, logits, slot_ids, token_mask, T, lse, p);
  });
  if (G > 1) hipLaunchKernelGGL(finish_kernel, dim3(1), dim3(NTHR), 0, s, p);
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
  const int per = GWAVES * tokens_per_wave(N);
  const int G = std::min((T + per - 1) / per, cu_count() * 8);
  by_width(N, [&](auto gl, auto kpl) {
    constexpr int GL = decltype(gl)::value, KPL = decltype(kpl)::value;
    if (dtype == MOE_F32)
      hipLaunchKernelGGL((grad_kernel<GL, KPL, float>), dim3(G), dim3(GNTHR), 0, s, logits,
                         topk_ids, token_mask, lse, counts, d_losses, d_gates, T, N, k,
                         static_cast<float*>(dlogits));
    else
      hipLaunchKernelGGL((grad_kernel<GL, KPL, __bf16>), dim3(G), dim3(GNTHR), 0, s, logits,
                         topk_ids, token_mask, lse, counts, d_losses, d_gates, T, N, k,
                         static_cast<__bf16*>(dlogits));
  });
  return launch_status();
}
