// moe_grad_table and moe_grad_clip: the norm of many gradient tensors together
// and their scaling to a largest norm.
//
//   norm = sqrt(sum g^2);   out = g min(1, max_norm / norm)
//
// Tensors are cut into blocks of 16 KB, counted from their address rounded down
// to 16 bytes, and a workgroup takes a contiguous run of blocks, whatever
// tensors they belong to: one launch for the squares and one for the scaling,
// for any number and mixture of tensors.  Bound by HBM (gradients read twice,
// written once).  Squares are fp64 from the first term: exact products, no
// overflow anywhere in the types' ranges.
//
// Measured: 1.22 GB of bf16 gradients 253 us for the squares (4.8 TB/s) and 476 for
// the scaling (5.1 TB/s); 240 tensors of 202 MB 40 and 70.
#include <algorithm>
#include <vector>

#include "common.h"
#include "linear_common.h"

namespace moe {
namespace clip {

constexpr int NTHR = 256;
constexpr int BLOCK = 16384;  // bytes of a block
constexpr int WORDS = MOE_GRAD_TABLE_WORDS;
// row of the table: address, output address, first block << 1 | bf16, elements;
// behind the last tensor a row whose first block is their number

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct Tensor {
  uint64_t in, out;  // addresses
  int64_t first;     // its first block
  bool bf16;
  int64_t elements;
};

__device__ __forceinline__ int64_t first_of(const int64_t* table, int i) {
  return table[static_cast<size_t>(i) * WORDS + 2] >> 1;
}

// The last tensor whose first block is at most b (tensors of no blocks are passed over).
__device__ __forceinline__ int find(const int64_t* table, int n, int64_t b) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (first_of(table, mid) <= b) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ Tensor read(const int64_t* table, int i) {
  const int64_t* p = table + static_cast<size_t>(i) * WORDS;
  return {static_cast<uint64_t>(p[0]), static_cast<uint64_t>(p[1]), p[2] >> 1, (p[2] & 1) != 0, p[3]};
}

__device__ __forceinline__ double square(float f) {
  const double d = static_cast<double>(f);
  return d * d;
}

// The workgroup's blocks
struct Run {
  int64_t lo, hi;
};
__device__ __forceinline__ Run run_of(int64_t blocks) {
  return {blocks * blockIdx.x / gridDim.x, blocks * (blockIdx.x + 1) / gridDim.x};
}

// The values of one element at address p
__device__ __forceinline__ float element(uint64_t p, bool bf16) {
  return bf16 ? __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p)) << 16)
              : *reinterpret_cast<const float*>(p);
}

constexpr int PIECES = BLOCK / 16 / NTHR;  // 16-byte pieces of a thread in a block

// s: two running sums
__device__ __forceinline__ void add_squares(u32x4 v, bool bf16, double* s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      s[0] += square(__uint_as_float(v[i] << 16));
      s[1] += square(__uint_as_float(v[i] & 0xffff0000u));
    } else {
      s[i % 2] += square(__uint_as_float(v[i]));
    }
  }
}

__global__ __launch_bounds__(NTHR) void squares_kernel(const int64_t* __restrict__ table, int n,
                                                       int64_t blocks, double* __restrict__ part) {
  __shared__ double red[NTHR / MOE_WAVE];
  const Run run = run_of(blocks);
  double s[2] = {};
  int i = run.lo < run.hi ? find(table, n, run.lo) : 0;
  for (int64_t b = run.lo; b < run.hi; ++b) {
    while (first_of(table, i + 1) <= b) ++i;
    const Tensor t = read(table, i);
    const int size = t.bf16 ? 2 : 4;
    const uint64_t end = t.in + static_cast<uint64_t>(t.elements) * size;
    const uint64_t base = (t.in & ~uint64_t(15)) + static_cast<uint64_t>(b - t.first) * BLOCK;
    const uint64_t mine = base + threadIdx.x * 16;
    if (base >= t.in && base + BLOCK <= end) {  // all loads of a whole block at once
      u32x4 v[PIECES];
#pragma unroll
      for (int j = 0; j < PIECES; ++j) v[j] = *reinterpret_cast<const u32x4*>(mine + j * NTHR * 16);
#pragma unroll
      for (int j = 0; j < PIECES; ++j) add_squares(v[j], t.bf16, s);
      continue;
    }
    for (int j = 0; j < PIECES; ++j) {
      const uint64_t p = mine + j * NTHR * 16;
      if (p >= t.in && p + 16 <= end) {
        add_squares(*reinterpret_cast<const u32x4*>(p), t.bf16, s);
      } else {
        for (uint64_t q = p; q < p + 16; q += size)
          if (q >= t.in && q < end) s[0] += square(element(q, t.bf16));
      }
    }
  }
  double sum = s[0] + s[1];
  sum = wave_sum_f64(sum);
  if (lane_id() == 0) red[threadIdx.x / MOE_WAVE] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0;
    for (int w = 0; w < NTHR / MOE_WAVE; ++w) sum += red[w];
    part[blockIdx.x] = sum;
  }
}

// Sum of the workgroups' squares, in every thread.
__device__ __forceinline__ double join(const double* part, int parts) {
  __shared__ double red[NTHR / MOE_WAVE];
  double v = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < parts; i += NTHR) v += part[i];
  v = wave_sum_f64(v);
  if (lane_id() == 0) red[threadIdx.x / MOE_WAVE] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < NTHR / MOE_WAVE; ++w) v += red[w];
  return v;
}

__global__ __launch_bounds__(NTHR) void norm_kernel(const double* __restrict__ part, int parts,
                                                    float* norm) {
  const double v = join(part, parts);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(v));
}

// f times m 2^e: the factor keeps its digits where it lies below fp32's normal
// range (gradients whose norm is beyond 2^126).
struct Factor {
  float m;
  int e;
  __device__ __forceinline__ float operator()(float f) const { return ldexpf(f * m, e); }
};

__global__ __launch_bounds__(NTHR) void scale_kernel(const int64_t* __restrict__ table, int n,
                                                     int64_t blocks,
                                                     const double* __restrict__ part, int parts,
                                                     double max_norm, float* norm) {
  const double v = sqrt(join(part, parts));
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(v);
  const bool keep = !(v > max_norm && v < INFINITY);
  Factor c{1.f, 0};
  if (!keep) c.m = static_cast<float>(frexp(max_norm / v, &c.e));
  // Last block first: what the squares read last is still in the last-level cache.
  const Run run = run_of(blocks);
  int i = run.lo < run.hi ? find(table, n, run.hi - 1) : 0;
  for (int64_t b = run.hi - 1; b >= run.lo; --b) {
    while (first_of(table, i) > b) --i;
    const Tensor t = read(table, i);
    if (keep && t.in == t.out) continue;
    const int size = t.bf16 ? 2 : 4;
    const uint64_t end = t.in + static_cast<uint64_t>(t.elements) * size;
    const uint64_t base = (t.in & ~uint64_t(15)) + static_cast<uint64_t>(b - t.first) * BLOCK;
    const uint64_t mine = base + threadIdx.x * 16, move = t.out - t.in;
    auto scaled = [&](u32x4 w) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = t.bf16 ? lin::pack2(c(__uint_as_float(w[k] << 16)),
                                   c(__uint_as_float(w[k] & 0xffff0000u)))
                      : __float_as_uint(c(__uint_as_float(w[k])));
      return w;
    };
    if (base >= t.in && base + BLOCK <= end) {
      u32x4 v[PIECES];
#pragma unroll
      for (int j = 0; j < PIECES; ++j) v[j] = *reinterpret_cast<const u32x4*>(mine + j * NTHR * 16);
#pragma unroll
      for (int j = 0; j < PIECES; ++j)
        *reinterpret_cast<u32x4*>(mine + move + j * NTHR * 16) = scaled(v[j]);
      continue;
    }
    for (int j = 0; j < PIECES; ++j) {
      const uint64_t p = mine + j * NTHR * 16;
      if (p >= t.in && p + 16 <= end) {
        *reinterpret_cast<u32x4*>(p + move) = scaled(*reinterpret_cast<const u32x4*>(p));
      } else {
        for (uint64_t q = p; q < p + 16; q += size)
          if (q >= t.in && q < end) {
            const float f = c(element(q, t.bf16));
            if (t.bf16) lin::store1(reinterpret_cast<uint16_t*>(q + move), f);
            else lin::store1(reinterpret_cast<float*>(q + move), f);
          }
      }
    }
  }
}

// Workgroups: eight to a CU.
inline int grid_of(int64_t blocks) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(blocks, 8 * cu_count())));
}

struct Span {
  uint64_t lo, hi;
  int i;
  bool operator<(const Span& o) const { return lo < o.lo; }
};

}  // namespace clip
}  // namespace moe

using namespace moe;
using namespace moe::clip;

extern "C" int moe_grad_table(const void* const* grads, void* const* outs, const int64_t* elements,
                              const int32_t* dtypes, int n, int64_t* table, int64_t* blocks) try {
  if (n < 0 || n > (1 << 20) || !table || !blocks ||
      (n > 0 && (!grads || !outs || !elements || !dtypes)))
    return MOE_EINVAL;
  std::vector<Span> out;
  int64_t first = 0;
  for (int i = 0; i < n; ++i) {
    if (dtypes[i] != MOE_F32 && dtypes[i] != MOE_BF16) return MOE_EUNSUP;
    const int64_t size = dtypes[i] == MOE_BF16 ? 2 : 4;
    const uint64_t a = reinterpret_cast<uint64_t>(grads[i]), o = reinterpret_cast<uint64_t>(outs[i]);
    if (elements[i] < 0 || elements[i] > (int64_t(1) << 40)) return MOE_EINVAL;
    if (elements[i] > 0 && (!a || !o || a % size || o % size || a % 16 != o % 16)) return MOE_EINVAL;
    int64_t* row = table + static_cast<size_t>(i) * WORDS;
    row[0] = static_cast<int64_t>(a);
    row[1] = static_cast<int64_t>(o);
    row[2] = first * 2 + (dtypes[i] == MOE_BF16);
    row[3] = elements[i];
    if (elements[i] > 0) {
      const int64_t bytes = elements[i] * size;
      out.push_back({o, o + bytes, i});
      first += (static_cast<int64_t>(a % 16) + bytes + BLOCK - 1) / BLOCK;
    }
  }
  int64_t* last = table + static_cast<size_t>(n) * WORDS;
  last[0] = last[1] = last[3] = 0;
  last[2] = first * 2;
  *blocks = first;
  std::sort(out.begin(), out.end());
  for (size_t j = 1; j < out.size(); ++j)
    if (out[j].lo < out[j - 1].hi) return MOE_EINVAL;
  for (int i = 0; i < n; ++i) {  // a gradient and the outputs that reach into it
    if (elements[i] == 0) continue;
    const uint64_t a = reinterpret_cast<uint64_t>(grads[i]);
    const uint64_t end = a + elements[i] * (dtypes[i] == MOE_BF16 ? 2 : 4);
    auto it = std::lower_bound(out.begin(), out.end(), Span{end, 0, 0});
    if (it == out.begin()) continue;
    --it;  // the last output that starts before the gradient's end
    if (it->hi > a && !(it->i == i && it->lo == a)) return MOE_EINVAL;
  }
  return MOE_OK;
} catch (...) {  // out of host memory
  return MOE_EINVAL;
}

extern "C" size_t moe_grad_clip_workspace_size(int64_t blocks) {
  return blocks < 0 ? 0 : static_cast<size_t>(grid_of(blocks)) * sizeof(double) + 256;
}

extern "C" int moe_grad_clip(const int64_t* table, int n, int64_t blocks, double max_norm,
                             float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  if (n < 0 || n > (1 << 20) || blocks < 0 || !(max_norm > 0.0) || !norm || !table || !workspace ||
      reinterpret_cast<uintptr_t>(workspace) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(table) % 8 != 0 || (n == 0 && blocks > 0) ||
      workspace_bytes < moe_grad_clip_workspace_size(blocks))
    return MOE_EINVAL;
  hipStream_t s = as_stream(stream);
  const int g = grid_of(blocks);
  double* part = static_cast<double*>(workspace);
  hipLaunchKernelGGL(squares_kernel, dim3(g), dim3(NTHR), 0, s, table, n, blocks, part);
  if (max_norm < INFINITY)
    hipLaunchKernelGGL(scale_kernel, dim3(g), dim3(NTHR), 0, s, table, n, blocks, part, g, max_norm,
                       norm);
  else
    hipLaunchKernelGGL(clip::norm_kernel, dim3(1), dim3(NTHR), 0, s, part, g, norm);
  return launch_status();
}
