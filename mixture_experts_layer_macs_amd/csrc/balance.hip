// moe_balance_loss and moe_router_backward: the router's training losses and
// the gradient of its logits.
//
// With p = softmax(z_t), c_j the slots that name expert j, n the unmasked
// tokens and lse_t = log sum_j exp z_tj,
//   balance = N / (k n) sum_j c_j P_j,   P_j = (1/n) sum_t p_tj
//   z loss  = (1/n) sum_t lse_t^2
//   dz_tj   = p_tj (u_tj - sum_i p_ti u_ti) + dL/dz_loss 2 lse_t p_tj / n,
//   u_tj    = dL/dbalance N c_j / (k n^2) + sum_{s: id_ts = j} dL/dgate_ts
// (the counts carry no gradient).  Both passes read the logits once, a token's
// N logits in the registers of a group of 8 to 64 lanes.  Sums over tokens are
// fp64 from the first term on, in a fixed order (the additions run beside the
// loads: fp32 runs of 32 tokens were no faster).
//
// Measured: 65521 tokens, 256 experts: loss 22.2 us (67 MB, 3.0 TB/s) and 9.8
// for the second launch, gradient 34.0 us (134 MB, 3.9 TB/s); a large copy
// runs at 4.8 TB/s.  128 tokens, 128 experts: 8.6 and 4.0 us, latency.
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
  return v;
}
template <int GL>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr (GL == MOE_WAVE) return wave_sum(v);
  return group_reduce<float, GL>(v, [](float a, float b) { return a + b; });
}
template <int GL>
__device__ __forceinline__ float group_max(float v) {
  if constexpr (GL == MOE_WAVE) return wave_max(v);
  return group_reduce<float, GL>(v, [](float a, float b) { return fmaxf(a, b); });
}

// Partial sums of the workgroups, in the workspace, and the outputs.
struct Part {
  double* zsq;     // [G]
  double* prob;    // [G][pitch], zeros behind column N
  int32_t* count;  // [G][pitch]
  int32_t* n;      // [G]
  float *losses, *mean_prob;
  int32_t* counts;
  int G, N, k, pitch;  // pitch: N rounded up to 4
};

// The losses from sum_j c_j P_j (dot), sum_t lse^2 and n.
__device__ __forceinline__ void write_losses(const Part& p, double dot, double zsq, int n) {
  const double inv = n > 0 ? 1.0 / n : 0.0;
  p.losses[0] = static_cast<float>(dot * inv * p.N / p.k);
  p.losses[1] = static_cast<float>(zsq * inv);
  p.counts[p.N] = n;
}

// Sum of one value per thread of the workgroup, in thread 0.
__device__ __forceinline__ double block_sum(double v, double* red) {
  v = wave_sum_f64(v);
  __syncthreads();
  if (lane_id() == 0) red[threadIdx.x / MOE_WAVE] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < WAVES; ++w) s += red[w];
  return s;
}

// The workgroups' sums to the outputs, one workgroup: a thread owns four
// columns of every R-th partial row, 8 rows in flight.  What it reads was
// written on other XCDs, so a dependent round costs a trip to memory (one
// column per thread and as many rounds took 23 us at G = N = 256; now 9.8, what
// one CU takes to read 768 KB.  Parts rounded to fp32 took 6.9).
__global__ __launch_bounds__(NTHR) void finish_kernel(Part p) {
  __shared__ double s_p[NTHR][4];
  __shared__ int s_c[NTHR][4];
  __shared__ double red[WAVES], s_z;
  __shared__ int s_n;
  typedef double f64x2 __attribute__((ext_vector_type(2)));  // the workspace starts at 16 bytes
  typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
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
  int quads = 4;  // threads along the columns: a power of two that covers N / 4
  while (quads * 4 < p.N) quads *= 2;
  const int R = NTHR / quads, c = (tid & (quads - 1)) * 4, r = tid / quads;
  double sum[4] = {};
  int count[4] = {};
  if (c < p.N) {
    for (int g0 = r; g0 < p.G; g0 += 8 * R) {
      f64x2 f[8][2];
      i32x4 m[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const size_t at = static_cast<size_t>(min(g0 + u * R, p.G - 1)) * p.pitch + c;
        f[u][0] = *reinterpret_cast<const f64x2*>(p.prob + at);
        f[u][1] = *reinterpret_cast<const f64x2*>(p.prob + at + 2);
        m[u] = *reinterpret_cast<const i32x4*>(p.count + at);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const bool in = g0 + u * R < p.G;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[i] += in ? f[u][i / 2][i % 2] : 0.0;
          count[i] += in ? m[u][i] : 0;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s_p[tid][i] = sum[i];
    s_c[tid][i] = count[i];
  }
  __syncthreads();
  const int n = s_n;
  const double inv = n > 0 ? 1.0 / n : 0.0;
  double dot = 0.0;
  if (tid < p.N) {
    double v = 0.0;
    int m = 0;
    for (int i = 0; i < R; ++i) {  // the same order every time
      v += s_p[i * quads + tid / 4][tid % 4];
      m += s_c[i * quads + tid / 4][tid % 4];
    }
    v *= inv;
    p.counts[tid] = m;
    p.mean_prob[tid] = static_cast<float>(v);
    dot = v * m;
  }
  dot = block_sum(dot, red);
  if (tid == 0) write_losses(p, dot, s_z, n);
}

// A row whose logits are all -inf has no probabilities: it counts as a token
// and adds nothing else.  The logits of the next D tokens are in flight while
// one is worked on: a short batch is a chain of memory latencies otherwise
// (one token ahead took 10.8 us for 128 tokens, 128 experts).
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
  const int lane = lane_id(), gl = lane & (GL - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
  // the token of a lane's group; GL == 64: the same for the wave, in scalar registers
  const int sub = GL == MOE_WAVE ? 0 : lane / GL;
  for (int j = threadIdx.x; j < N; j += NTHR) s_count[j] = 0;
  __syncthreads();
  constexpr int D = KPL <= 4 ? 4 : KPL <= 8 ? 2 : 1;
  float znext[D][KPL];
  double pd[KPL] = {}, zsq = 0.0;
  int n = 0, idnext[D];
  uint32_t onnext[D];
  // every load of a request is unconditional (a branch around one waits for
  // all that are in flight): without a mask, bytes that are not looked at
  const uint8_t* mask_or_any = mask ? mask : reinterpret_cast<const uint8_t*>(logits);
  const int step = gridDim.x * WAVES * TPW;
  auto request = [&](int t, int d) {
    const int u = min(t, T - 1);  // past the end: a token that is not used
    onnext[d] = mask_or_any[u];
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int j = gl + GL * i;
      znext[d][i] = logits[static_cast<size_t>(u) * N + min(j, N - 1)];
    }
    idnext[d] = ids[static_cast<size_t>(u) * k + min(gl, k - 1)];
  };
  auto work = [&](int t, int d) {
    float z[KPL], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < KPL; ++i) z[i] = gl + GL * i < N ? znext[d][i] : -INFINITY;
    int id = idnext[d];
    const bool on = t < T && (mask == nullptr || onnext[d] != 0);
    request(t + D * step, d);
#pragma unroll
    for (int i = 0; i < KPL; ++i) top = fmaxf(top, z[i]);
    if (on) {
      for (int s = gl; s < k; s += GL) {
        if (s >= GL) id = ids[static_cast<size_t>(t) * k + s];
        if (static_cast<unsigned>(id) < static_cast<unsigned>(N)) atomicAdd(&s_count[id], 1);
      }
    }
    top = group_max<GL>(top);
    // the maximum passes over NaN: a row of NaN is told from one of -inf by its
    // sum, NaN and 0 with a finite shift
    const float shift = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      z[i] = __expf(z[i] - shift);
      sum += z[i];
    }
    sum = group_sum<GL>(sum);
    const bool some = on && sum != 0.f;
    // hardware exponential, reciprocal and logarithm, a unit or two of fp32 each:
    // lse and the probabilities end 1.1e-7 off
    const float inv = __builtin_amdgcn_rcpf(sum), l = shift + __logf(sum);
    if (some) {  // padding may hold NaN
#pragma unroll
      for (int i = 0; i < KPL; ++i) pd[i] += z[i] * inv;
      zsq += static_cast<double>(l) * l;
    }
    n += on;
    if (gl == 0 && t < T) lse[t] = some ? l : on ? -INFINITY : 0.f;
  };
  const int t0 = (blockIdx.x * WAVES + wave) * TPW;
  if (T > 0) {
#pragma unroll
    for (int d = 0; d < D; ++d) request(t0 + sub + d * step, d);
    for (int tb = t0; tb < T; tb += D * step)
#pragma unroll
      for (int d = 0; d < D; ++d) work(tb + sub + d * step, d);
  }
  if (gl != 0) {  // every lane of a group counted its tokens
    zsq = 0.0;
    n = 0;
  }
#pragma unroll
  for (int i = 0; i < KPL; ++i)
    for (int m = GL; m < MOE_WAVE; m *= 2) pd[i] += __shfl_xor(pd[i], m, MOE_WAVE);
  zsq = wave_sum_f64(zsq);
  n = wave_sum(n);
  if (lane == 0) {
    s_z[wave] = zsq;
    s_n[wave] = n;
  }
  __syncthreads();
  double zall = 0.0;
  int nall = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    zall += s_z[w];
    nall += s_n[w];
  }
  const bool alone = gridDim.x == 1;  // a short batch: one workgroup, one launch
  const double invn = nall > 0 ? 1.0 / nall : 0.0;
  const size_t g = blockIdx.x;
  constexpr int PER = COLS / GL;  // registers of a wave per round
  double dot = 0.0;
#pragma unroll
  for (int i0 = 0; i0 < KPL; i0 += PER) {
    __syncthreads();
#pragma unroll
    for (int i = i0; i < i0 + PER && i < KPL; ++i)
      if (lane < GL) s_prob[wave][(i - i0) * GL + gl] = pd[i];
    __syncthreads();
    const int j = i0 * GL + threadIdx.x;
    if (threadIdx.x >= COLS || threadIdx.x >= (KPL - i0) * GL || j >= part.pitch) continue;
    double v = 0.0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += s_prob[w][threadIdx.x];
    const int c = j < N ? s_count[j] : 0;
    if (alone && j < N) {
      part.mean_prob[j] = static_cast<float>(v * invn);
      part.counts[j] = c;
      dot += v * invn * c;
    } else if (!alone) {
      part.prob[g * part.pitch + j] = j < N ? v : 0.0;
      part.count[g * part.pitch + j] = c;
    }
  }
  if (alone) {
    dot = block_sum(dot, s_z);
    if (threadIdx.x == 0) write_losses(part, dot, zall, nall);
  } else if (threadIdx.x == 0) {
    part.zsq[g] = zall;
    part.n[g] = nall;
  }
}

__device__ __forceinline__ void store_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_elem(__bf16* p, float v) { *p = static_cast<__bf16>(v); }

constexpr int GNTHR = 256, GWAVES = GNTHR / MOE_WAVE;

// Slot q of a token sits in lane q of its group.  With GL == 64 a slot is read
// into scalar registers and touches only the register that holds its expert.
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
  const int sub = GL == MOE_WAVE ? 0 : lane / GL;
  const int step = gridDim.x * GWAVES * TPW, t0 = (blockIdx.x * GWAVES + wave) * TPW;
  // unconditional loads, as above; without d_gates, values that are not used
  const uint8_t* mask_or_any = mask ? mask : reinterpret_cast<const uint8_t*>(logits);
  const int32_t* id_or_any = d_gates ? ids : reinterpret_cast<const int32_t*>(logits);
  const float* dg_or_any = d_gates ? d_gates : logits;
  float znext[KPL], lnext, dgnext;
  int idnext;
  uint32_t onnext;
  auto request = [&](int t) {
    const int u = min(t, T - 1);  // past the end: a token that is not used
    onnext = mask_or_any[u];
    lnext = lse[u];
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      znext[i] = logits[static_cast<size_t>(u) * N + min(gl + GL * i, N - 1)];
    // k <= N: the substitute's T x k elements lie inside the logits
    idnext = id_or_any[static_cast<size_t>(u) * k + min(gl, k - 1)];
    dgnext = dg_or_any[static_cast<size_t>(u) * k + min(gl, k - 1)];
  };
  request(t0 + sub);
  for (int tb = t0; tb < T; tb += step) {
    const int t = tb + sub;
    const float l = lnext;
    const bool on = (mask == nullptr || onnext != 0) && l != -INFINITY;
    int id = idnext;
    float dg = dgnext;
    float p[KPL], u[KPL];
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      p[i] = gl + GL * i < N ? __expf(znext[i] - l) : 0.f;
      u[i] = base[i];
    }
    request(t + step);
    if (d_gates) {
      if constexpr (GL == MOE_WAVE) {
        for (int s0 = 0; s0 < k; s0 += MOE_WAVE) {
          if (s0 > 0) {  // more than 64 slots
            const bool in = s0 + lane < k;
            id = in ? ids[static_cast<size_t>(tb) * k + s0 + lane] : -1;
            dg = in ? d_gates[static_cast<size_t>(tb) * k + s0 + lane] : 0.f;
          }
          const int m = min(MOE_WAVE, k - s0);
#pragma unroll 4
          for (int q = 0; q < m; ++q) {
            const int e = read_lane(id, q);
            if (static_cast<unsigned>(e) >= static_cast<unsigned>(N)) continue;
            const float d = __uint_as_float(read_lane(__float_as_uint(dg), q));
            const float mine = lane == (e & 63) ? d : 0.f;
#pragma unroll
            for (int i = 0; i < KPL; ++i)
              if (KPL == 1 || (e >> 6) == i) u[i] += mine;
          }
        }
      } else {  // k <= N <= GL
        for (int q = 0; q < k; ++q) {
          const int from = (lane & ~(GL - 1)) + q;
          const int e = __shfl(id, from, MOE_WAVE);
          const float d = __shfl(dg, from, MOE_WAVE);
          u[0] += e == gl && e < N ? d : 0.f;
        }
      }
    }
    // lse is rounded to fp32, which costs every p of a token the same factor, up
    // to |lse| 2^-24 off 1: the probabilities are those of the row's own sum
    float dot = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      dot += p[i] * u[i];
      sum += p[i];
    }
    const float inv_sum = __builtin_amdgcn_rcpf(group_sum<GL>(sum));
    const float shift = zc * l - group_sum<GL>(dot) * inv_sum;
    if (t < T) {
#pragma unroll
      for (int i = 0; i < KPL; ++i)
        if (gl + GL * i < N)
          store_elem(&dlogits[static_cast<size_t>(t) * N + gl + GL * i],
                     on ? p[i] * inv_sum * (u[i] + shift) : 0.f);
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

inline size_t up4(int n) { return (static_cast<size_t>(n) + 3) & ~size_t(3); }

inline size_t part_bytes(int G, int N) { return static_cast<size_t>(G) * (up4(N) * 12 + 12) + 64; }

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
  if (workspace_bytes < part_bytes(G, N) || reinterpret_cast<uintptr_t>(workspace) % 16 != 0)
    return MOE_EINVAL;
  Part p;
  p.pitch = static_cast<int>(up4(N));
  p.prob = static_cast<double*>(workspace);
  p.count = reinterpret_cast<int32_t*>(p.prob + static_cast<size_t>(G) * p.pitch);
  p.zsq = reinterpret_cast<double*>(p.count + static_cast<size_t>(G) * p.pitch);
  p.n = reinterpret_cast<int32_t*>(p.zsq + G);
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
