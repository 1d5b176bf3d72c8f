// bf16 matrix product on MFMA tiles for the dense layer:
//   C[m][n] = sum_k R(m, k) C(n, k),
// each operand either reduction-contiguous (its rows are m or n, as x and w of
// y = x w^T) or reduction-strided (its rows are k, as w of dz w and both
// operands of dz^T x).
//
// A slice of 64 k travels global -> LDS by direct-to-LDS loads of 1 KB per
// wave instruction, the row operand one slice ahead (2 stages) and the column
// operand two (3 stages).  Reduction-contiguous: LDS rows of 64 k, 16-byte
// chunk c of row r at c ^ ((r >> 1) & 7), fragments by 16-byte reads.
// Reduction-strided: LDS rows of the tile's m (or n), one per k; the fragments
// come through the transposing 8-byte LDS read, which hands lane i of 16 the
// column i of a 4 x 16 block, so no operand is ever transposed in memory.  A
// wave's read covers 64 bytes of four consecutive k; the 64-byte groups are
// XORed with k (below) so that the four fall on different banks.
//
// v_mfma_f32_32x32x16_bf16 with the column operand as A: a lane ends with four
// consecutive output columns of one row.
#pragma once

#include "common.h"
#include "dma.h"
#include "linear_common.h"

namespace moe {
namespace lin {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int SLICE = 64;  // k per ring stage

struct Mma {
  const uint16_t *r, *c;  // operands
  size_t ldr, ldc;        // elements between their stored rows
  int M, N, K;            // output rows and columns (GLU: columns of y), reduction
  int tm, tn;             // tiles along M and N
  int splits, per_split;  // slices of 64 k per split
  float* part;            // splits > 1: [splits][M][N] partial sums
  Epilogue e;
};

// One operand's share of a wave: Q loads of 1 KB per slice.
template <bool STRIDED, int EXT, int W>
struct Operand {
  static constexpr int Q = EXT / 8 / W;
  static constexpr int BYTES = EXT * SLICE * 2;
  static_assert(Q >= 1, "one load per wave at least");
  uint32_t voff[Q];
  int first[2];  // contiguous: k of the lane's chunk in the slice, by load parity
  i32x4 rsrc;    // contiguous: the tile's rows
  const char* base;
  size_t step;   // strided: bytes of a k row
  uint32_t tail; // strided: bytes from base to the end of a k row's used part

  // rows: valid rows from p (contiguous); cols: valid elements of a k row
  // from p (strided)
  __device__ __forceinline__ void init(const uint16_t* p, size_t ld, int valid, int wave,
                                       int lane) {
    if constexpr (!STRIDED) {
      const uint32_t row_bytes = static_cast<uint32_t>(ld) * 2;
      rsrc = buffer_rsrc(p, static_cast<uint32_t>(max(valid, 0)) * row_bytes);
      const int lrow = lane / 8, slot = lane % 8;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int row = (wave * Q + q) * 8 + lrow;
        const int ch = slot ^ ((row >> 1) & 7);
        if (q < 2) first[q] = ch * 8;
        voff[q] = row < valid ? static_cast<uint32_t>(row) * row_bytes + ch * 16 : OOB_OFF;
      }
      if (Q == 1) first[1] = first[0];
    } else {
      constexpr int CPR = EXT / 8, RPI = 64 / CPR;
      base = reinterpret_cast<const char*>(p);
      step = ld * 2;
      tail = static_cast<uint32_t>(max(valid, 0)) * 2;
      const int lrow = lane / CPR, slot = lane % CPR;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int row = (wave * Q + q) * RPI + lrow;
        const int ch = slot ^ swizzle(row);
        voff[q] = ch * 8 < valid ? static_cast<uint32_t>(row) * static_cast<uint32_t>(step) + ch * 16
                                 : OOB_OFF;
      }
    }
  }
  static __device__ __forceinline__ int swizzle(int k) {
    return EXT >= 128 ? (k & 3) << 2 : ((k >> 1) & 1) << 2;
  }
  // loads of the slice from k0 (k up to kend) into the stage at lds
  __device__ __forceinline__ void load(int k0, int kend, uint32_t lds, int wave) const {
    if constexpr (!STRIDED) {
      const int left = kend - k0;
#pragma unroll
      for (int q = 0; q < Q; ++q)
        lds_dma16(rsrc, first[q & 1] < left ? voff[q] : OOB_OFF, static_cast<uint32_t>(k0) * 2,
                  lds + (wave * Q + q) * 1024);
    } else {
      const uint32_t rows = static_cast<uint32_t>(min(SLICE, kend - k0));
      const i32x4 rs = buffer_rsrc(base + static_cast<size_t>(k0) * step,
                                   (rows - 1) * static_cast<uint32_t>(step) + tail);
#pragma unroll
      for (int q = 0; q < Q; ++q) lds_dma16(rs, voff[q], 0, lds + (wave * Q + q) * 1024);
    }
  }
};

// Fragment reader: 32 rows (m or n) x 16 k from row m0 of the operand's tile.
typedef __attribute__((address_space(3))) const unsigned char lds_cbyte;
template <bool STRIDED, int EXT>
struct Reader {
  static __device__ __forceinline__ uint32_t lane_off(int m0, int lane) {
    if constexpr (!STRIDED) {
      return (m0 + (lane & 31)) * (SLICE * 2);
    } else {
      const int g = lane >> 4, i = lane & 15;
      const int k = 8 * (g >> 1) + (i >> 2);
      const int ch = (m0 / 8 + 2 * (g & 1) + ((i & 3) >> 1)) ^ Operand<true, EXT, 1>::swizzle(k);
      return k * (EXT * 2) + ch * 16 + 8 * (i & 1);
    }
  }
  static __device__ __forceinline__ bf16x8 read(lds_cbyte* stage, uint32_t off, int kk, int lane) {
    if constexpr (!STRIDED) {
      typedef __attribute__((address_space(3))) const bf16x8 frag;
      const int sw = ((kk * 2 + (lane >> 5)) ^ (((lane & 31) >> 1) & 7)) << 4;
      return *(frag*)(stage + off + sw);
    } else {
      typedef __attribute__((address_space(3))) s16x4 quad;
      // k + 4 keeps the low two bits of k; its third bit does not enter the
      // 64-byte swizzle of extents of 128 and more, nor k >> 1 & 1
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((quad*)(stage + off + kk * 16 * EXT * 2));
      const s16x4 hi =
          __builtin_amdgcn_ds_read_tr16_b64_v4i16((quad*)(stage + off + (kk * 16 + 4) * EXT * 2));
      union {
        s16x4 h[2];
        bf16x8 v;
      } u;
      u.h[0] = lo;
      u.h[1] = hi;
      return u.v;
    }
  }
};

// Tiles that run side by side on one XCD (workgroups go round-robin over the
// 8 XCDs, so each gets one contiguous range of the list) form blocks of
// GROUP tile rows, which share the operands' slices in that XCD's L2.
__device__ __forceinline__ bool tile_of(const Mma& a, int& mt, int& nt, int& split) {
  constexpr int GROUP = 4;
  const int tiles = a.tm * a.tn, total = tiles * a.splits;
  const int p = blockIdx.x, q = (total + 7) / 8;
  const int L = (p % 8) * q + p / 8;
  if (L >= total) return false;
  split = L / tiles;
  const int t = L - split * tiles;
  const int band = t / (GROUP * a.tn), in = t - band * GROUP * a.tn;
  const int rows = min(GROUP, a.tm - band * GROUP);
  mt = band * GROUP + in % rows;
  nt = in / rows;
  return true;
}

template <bool RS, bool CS, int BM, int BN, int WM, int WN, bool GLU, bool PART, int WGS>
__global__ __launch_bounds__(WM * WN * MOE_WAVE)
__attribute__((amdgpu_waves_per_eu(WM * WN * WGS / 4, WM * WN * WGS / 4)))
void mma_kernel(Mma a) {
  extern __shared__ __align__(16) unsigned char smem[];
  static_assert(!GLU || (!CS && !PART), "pairs of gate and up rows: y = x w^T only");
  constexpr int W = WM * WN;
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  static_assert(!GLU || FN % 2 == 0, "gate and up fragments in one wave");
  constexpr int SA = 2, SB = 3;
  typedef Operand<RS, BM, W> Row;
  typedef Operand<CS, BN, W> Col;
  typedef Reader<RS, BM> RowR;
  typedef Reader<CS, BN> ColR;
  constexpr int B_BASE = SA * Row::BYTES;
  constexpr int KK = SLICE / 16;
  constexpr int NMF = FM * FN;
  constexpr int NFR = FM * (RS ? 2 : 1) + FN * (CS ? 2 : 1);  // LDS reads per 16 k

  int mt, nt, split;
  if (!tile_of(a, mt, nt, split)) return;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
  const int wm = wave / WN, wn = wave % WN;
  constexpr int NC = GLU ? BN / 2 : BN;  // output columns of the tile
  const int m0 = mt * BM, n0 = nt * NC;
  const int k_lo = split * a.per_split * SLICE;
  const int k_hi = min(a.K, k_lo + a.per_split * SLICE);
  const int nk = (k_hi - k_lo + SLICE - 1) / SLICE;

  Row row;
  Col col;
  row.init(a.r + (RS ? m0 : m0 * a.ldr), a.ldr, min(BM, a.M - m0), wave, lane);
  if constexpr (GLU) {
    // the first half of the tile's rows are gate rows, the second the up rows
    // of the same columns; a wave's loads lie in one half
    const int half = wave >= W / 2;
    col.init(a.c + (static_cast<size_t>(half) * a.N + n0) * a.ldc, a.ldc, min(NC, a.N - n0),
             wave - half * (W / 2), lane);
  } else {
    col.init(a.c + (CS ? n0 : n0 * a.ldc), a.ldc, min(BN, a.N - n0), wave, lane);
  }
  const uint32_t lds_base = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char*)(smem))));
  lds_cbyte* lds0 = (lds_cbyte*)(smem);

  // Requests past the last slice fetch it again into a stage that is not read
  // any more, so that every iteration issues the same number of loads.
  auto load_row = [&](int t) {
    row.load(k_lo + min(t, nk - 1) * SLICE, k_hi, lds_base + (t % SA) * Row::BYTES, wave);
  };
  auto load_col = [&](int t) {
    uint32_t at = lds_base + B_BASE + (t % SB) * Col::BYTES;
    int w = wave;
    if constexpr (GLU) {
      const int half = wave >= W / 2;
      at += half * (Col::BYTES / 2);
      w -= half * (W / 2);
    }
    col.load(k_lo + min(t, nk - 1) * SLICE, k_hi, at, w);
  };

  uint32_t ro[FM], co[FN];
#pragma unroll
  for (int x = 0; x < FM; ++x) ro[x] = RowR::lane_off(wm * TM + x * 32, lane);
#pragma unroll
  for (int y = 0; y < FN; ++y)
    co[y] = ColR::lane_off(GLU ? (y < FN / 2 ? wn * (TN / 2) + y * 32
                                             : BN / 2 + wn * (TN / 2) + (y - FN / 2) * 32)
                               : wn * TN + y * 32,
                           lane);
  f32x16 acc[FM][FN];
#pragma unroll
  for (int x = 0; x < FM; ++x)
#pragma unroll
    for (int y = 0; y < FN; ++y)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[x][y][r] = 0.f;
  bf16x8 fr[2][FM], fc[2][FN];
  auto read = [&](int t, int kk, bf16x8* pr, bf16x8* pc) {
    lds_cbyte* A = lds0 + (t % SA) * Row::BYTES;
    lds_cbyte* B = lds0 + B_BASE + (t % SB) * Col::BYTES;
#pragma unroll
    for (int x = 0; x < FM; ++x) pr[x] = RowR::read(A, ro[x], kk, lane);
#pragma unroll
    for (int y = 0; y < FN; ++y) pc[y] = ColR::read(B, co[y], kk, lane);
  };

  // Row slice t is requested in iteration t - 1 and column slice t in
  // iteration t - 2, after row slice t - 1: when at most the newest column
  // slice's loads are outstanding, both slices t have landed.
  load_row(0);
  load_col(0);
  load_col(1);
  for (int t = 0; t < nk; ++t) {
    wait_vmcnt<Col::Q>();
    wg_barrier();
    load_row(t + 1);
    load_col(t + 2);
    read(t, 0, fr[0], fc[0]);
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      if (kk + 1 < KK) read(t, kk + 1, fr[(kk + 1) & 1], fc[(kk + 1) & 1]);
#pragma unroll
      for (int x = 0; x < FM; ++x)
#pragma unroll
        for (int y = 0; y < FN; ++y)
          acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fc[kk & 1][y], fr[kk & 1][x],
                                                             acc[x][y], 0, 0, 0);
      if (kk == 0) {
        __builtin_amdgcn_sched_group_barrier(0x0020, Row::Q + Col::Q, 0);  // requests
        __builtin_amdgcn_sched_group_barrier(0x0100, NFR, 0);              // first reads
      }
      if (kk + 1 < KK) interleave_groups<NMF, NFR>();
      else __builtin_amdgcn_sched_group_barrier(0x0008, NMF, 0);
    }
  }
  wait_vmcnt<0>();  // no load may land after the workgroup ends

  const int half = lane >> 5;
#pragma unroll
  for (int x = 0; x < FM; ++x) {
    const int m = m0 + wm * TM + x * 32 + (lane & 31);
    if (m >= a.M) continue;
#pragma unroll
    for (int y = 0; y < (GLU ? FN / 2 : FN); ++y) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + wn * (GLU ? TN / 2 : TN) + y * 32 + 8 * q + 4 * half;
        if (n >= a.N) continue;
        float g[4], u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] = acc[x][y][4 * q + i];
          if constexpr (GLU) u[i] = acc[x][y + FN / 2][4 * q + i];
        }
        if constexpr (PART)
          *reinterpret_cast<f32x4*>(a.part + (static_cast<size_t>(split) * a.M + m) * a.N + n) =
              f32x4{g[0], g[1], g[2], g[3]};
        else
          finish4<uint16_t, GLU>(a.e, m, n, a.N, g, u);
      }
    }
  }
}

}  // namespace lin
}  // namespace moe
