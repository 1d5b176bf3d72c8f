// bf16 matrix product on MFMA tiles for the dense layer:
//   C[m][n] = sum_k R(m, k) C(n, k),
// each operand either reduction-contiguous (its rows are m or n, as x and w of
// y = x w^T) or reduction-strided (its rows are k, as w of dz w and both
// operands of dz^T x).
//
// A slice of 64 k travels global -> LDS by direct-to-LDS loads of 1 KB per
// wave instruction through a ring of 2 row-operand and 3 column-operand
// stages.  Reduction-contiguous: LDS rows of 64 k, their 16-byte chunks XORed
// with the row, fragments by 16-byte reads.  Reduction-strided: LDS rows
// of the tile's m (or n), one per k; the fragments come through the
// transposing 8-byte LDS read, which hands lane i of 16 the column i of a
// 4 x 16 block, so no operand is ever transposed in memory.  A wave's read
// covers 64 bytes of four consecutive k; the 64-byte groups are XORed with k
// (below) so that the four fall on different banks.
//
// v_mfma_f32_32x32x16_bf16 with the column operand as A: a lane ends with four
// consecutive output columns of one row.
//
// Bound by the matrix pipe at the clock that its power allows (1.6 to 1.75 GHz
// in a long product, 77 % of its cycles busy; what is left is waiting for the
// ring).  Measured: 8192 x 2048 -> 768 swiglu with z kept 47 us (1.10 PFLOP/s);
// 4096 x 4096 -> 14336 410 us (1.17 PFLOP/s; the library's plain product 406),
// 445 with gelu.
#pragma once

#include "common.h"
#include "dma.h"
#include "linear_common.h"

namespace moe {
namespace lin {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// A value that every lane has, in a scalar register from here on.  The vector
// unit computes some of them (a division by a run-time number), and the compiler
// then moves them where they are used; a load that reads a scalar register less
// than five wait states behind the vector instruction that wrote it may see the
// old value, and the compiler keeps that distance only for loads that it knows.
// What an inline load's resource and offset are made of passes through here where
// a kernel starts; the build fails on loads that come too close all the same.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
template <typename T>
__device__ __forceinline__ T* uniform(T* p) {
  const uint64_t b = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int>(b));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<int>(b >> 32));
  return reinterpret_cast<T*>(static_cast<uint64_t>(hi) << 32 | lo);
}

constexpr int SLICE = 64;        // k per ring stage
constexpr int SA = 2, SB = 3;    // stages of the row and the column operand
constexpr int WM = 2, WN = 2, W = WM * WN;  // waves of a workgroup along M and N

struct Mma {
  const uint16_t *r, *c;  // operands
  size_t ldr, ldc;        // elements between their stored rows
  int M, N, K;            // output rows and columns (GLU: columns of y), reduction
  int tm, tn;             // tiles along M and N
  int splits, per_split;  // reduction length of a split, whole slices
  float* part;            // splits > 1: [splits][M][N] partial sums
  Epilogue e;
};

// One operand's share of a wave: Q loads of 1 KB per slice.  MIX (the weights
// of a gated activation): every 32 tile rows are 16 gate rows and the 16 up
// rows of the same columns, so that a lane's accumulators r and r + 8 are a
// pair; a load of 8 rows lies in one half.
// SL: k of a slice, 64 or 32.
template <bool STRIDED, bool MIX, int EXT, int NW, int SL = SLICE>
struct Operand {
  static constexpr int BYTES = EXT * SL * 2;
  static constexpr int RPL = 512 / SL, CPR = STRIDED ? EXT / 8 : SL / 8;  // contiguous: rows of a load; chunks of an LDS row
  static constexpr int Q = BYTES / 1024 / NW;
  static_assert(Q >= 1 && BYTES % (1024 * NW) == 0, "whole loads per wave");
  static_assert(STRIDED || SL == 32 || Q % 2 == 0, "rows of a load: the swizzle goes by its parity");
  static_assert(!(STRIDED && MIX), "gated weights are reduction-contiguous");
  uint32_t voff[Q];
  int first[2];  // contiguous: k of the lane's chunk in the slice, by load parity
  i32x4 rsrc, rsrc_up;  // contiguous: the tile's rows (MIX: gate, up); strided: the slice
  const char* base;
  uint32_t step; // strided: bytes of a k row
  uint32_t tail; // strided: bytes from base to the end of a k row's used part

  // valid: rows from p (contiguous), or elements of a k row from p (strided);
  // up: distance of the up rows in elements (MIX; valid counts the columns)
  __device__ __forceinline__ void init(const uint16_t* p, size_t ld, int valid, int wave, int lane,
                                       size_t up = 0) {
    if constexpr (!STRIDED) {
      const uint32_t row_bytes = static_cast<uint32_t>(ld) * 2;
      const uint32_t bytes = static_cast<uint32_t>(valid) * row_bytes;
      rsrc = buffer_rsrc(p, bytes);
      if constexpr (MIX) rsrc_up = buffer_rsrc(p + up, bytes);
      const int lrow = lane / CPR, slot = lane % CPR;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int row = (wave * Q + q) * RPL + lrow;
        const int ch = slot ^ row_swizzle(row);
        const int at = MIX ? row / 32 * 16 + row % 16 : row;
        if (q < 2) first[q] = ch * 8;
        voff[q] = at < valid ? static_cast<uint32_t>(at) * row_bytes + ch * 16 : OOB_OFF;
      }
    } else {
      base = uniform(reinterpret_cast<const char*>(p));
      step = uniform(static_cast<int>(ld * 2));
      tail = uniform(valid * 2);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int at = (wave * Q + q) * 64 + lane, row = at / CPR;
        const int ch = at % CPR ^ swizzle(row);
        voff[q] = ch * 8 < valid ? static_cast<uint32_t>(row) * step + ch * 16
                                 : OOB_OFF;
      }
    }
  }
  // Contiguous: 16-byte chunks of a row, so that 16 rows of a fragment read
  // cover all banks.
  static __device__ __forceinline__ int row_swizzle(int row) {
    return SL == 64 ? (row >> 1) & 7 : (row >> 2) & 3;
  }
  // Strided: the four k rows of a read, 64-byte group g of each: on different groups
  // of 16 banks.  LDS rows of 512 or 256 bytes start at bank 0, those of 384
  // (and 128) bytes at bank 0 and 32 in turn.
  static __device__ __forceinline__ int swizzle(int k) {
    return EXT % 128 == 0 ? (k & 3) << 2 : ((k >> 1) & 1) << 2;
  }
  // before the loads of the slice from k0 (k up to kend)
  __device__ __forceinline__ void fetch(int k0, int kend) {
    if constexpr (STRIDED) {
      const uint32_t rows = static_cast<uint32_t>(min(SL, kend - k0));
      rsrc = buffer_rsrc(base + static_cast<size_t>(k0) * step, (rows - 1) * step + tail);
    }
  }
  // load q of that slice into the stage at lds
  __device__ __forceinline__ void load(int q, int k0, int kend, uint32_t lds, int wave) const {
    if constexpr (!STRIDED) {
      lds_dma16(MIX && ((wave * Q + q) / (16 / RPL) & 1) ? rsrc_up : rsrc,
                first[q & 1] < kend - k0 ? voff[q] : OOB_OFF, static_cast<uint32_t>(k0) * 2,
                lds + (wave * Q + q) * 1024);
    } else {
      lds_dma16(rsrc, voff[q], 0, lds + (wave * Q + q) * 1024);
    }
  }
};

// Fragment reader: 32 rows (m or n) x 16 k from row m0 of the operand's tile.
typedef __attribute__((address_space(3))) const unsigned char lds_cbyte;
template <bool STRIDED, int EXT, int SL = SLICE>
struct Reader {
  typedef Operand<STRIDED, false, EXT, 1, SL> Op;
  static __device__ __forceinline__ uint32_t lane_off(int m0, int lane) {
    if constexpr (!STRIDED) {
      return (m0 + (lane & 31)) * (SL * 2);
    } else {
      const int g = lane >> 4, i = lane & 15;
      const int k = 8 * (g >> 1) + (i >> 2);
      const int ch = (m0 / 8 + 2 * (g & 1) + ((i & 3) >> 1)) ^ Op::swizzle(k);
      return k * (EXT * 2) + ch * 16 + 8 * (i & 1);
    }
  }
  static __device__ __forceinline__ bf16x8 read(lds_cbyte* stage, uint32_t off, int kk, int lane) {
    if constexpr (!STRIDED) {
      typedef __attribute__((address_space(3))) const bf16x8 frag;
      const int sw = ((kk * 2 + (lane >> 5)) ^ Op::row_swizzle(lane & 31)) << 4;
      return *(frag*)(stage + off + sw);
    } else {
      typedef __attribute__((address_space(3))) s16x4 quad;
      // the swizzle looks at the low two bits of k, which k + 4 and k + 16 keep
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
__device__ __forceinline__ bool tile_of(const Mma& a, int p, int& mt, int& nt, int& split) {
  constexpr int GROUP = 4;
  const int tiles = a.tm * a.tn, total = tiles * a.splits;
  const int q = (total + 7) / 8;
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

// Output staging: XC of a wave's row fragments at once, as fp32 rows padded by
// 16 bytes, within the ring's LDS.
template <int BM, int BN, int RING>
struct Staging {
  static constexpr int FM = BM / WM / 32, PITCH = BN + 4;
  static constexpr int XC = FM % 2 == 0 && WM * 2 * 32 * PITCH * 4 <= RING ? 2 : 1;
  static_assert(WM * XC * 32 * PITCH * 4 <= RING, "fits the ring");
};

// One tile: the sum over k_lo <= k < k_hi (not empty) of the operands' slices,
// whose chunks of V output columns go to out(row, column, sums, up sums), places
// within the tile, also those past the matrix's end.  Row and Col: Operand, or
// another with its functions; smem: LDS bytes, the ring.
template <bool RS, bool CS, int BM, int BN, bool GLU, int V, int SL = SLICE, int SA = lin::SA,
          int SB = lin::SB, int LDS = (SA * BM + SB * BN) * SL * 2, class Row, class Col, class Out>
__device__ __forceinline__ void mma_core(Row& row, Col& col, int k_lo, int k_hi,
                                         unsigned char* smem, Out out_chunk) {
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  static_assert(TM % 32 == 0 && TN % 32 == 0, "whole fragments");
  static_assert(SA >= 2 && SA <= 3 && SB == 3, "the order of requests, below");
  typedef Reader<RS, BM, SL> RowR;
  typedef Reader<CS, BN, SL> ColR;
  constexpr int B_BASE = SA * Row::BYTES;
  constexpr int KK = SL / 16;
  static_assert(KK % 2 == 0, "fragment sets alternate");
  constexpr int NMF = FM * FN;

  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
  const int wm = wave / WN, wn = wave % WN;
  constexpr int NC = GLU ? BN / 2 : BN;  // output columns of the tile
  const int nk = (k_hi - k_lo + SL - 1) / SL;
  const uint32_t lds_base = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char*)(smem))));
  lds_cbyte* lds0 = (lds_cbyte*)(smem);

  // Requests past the last slice fetch it again into a stage that is not read
  // any more, so that every iteration issues the same number of loads.
  auto load_row = [&](int t, int q) {
    row.load(q, k_lo + min(t, nk - 1) * SL, k_hi, lds_base + (t % SA) * Row::BYTES, wave);
  };
  auto load_col = [&](int t, int q) {
    col.load(q, k_lo + min(t, nk - 1) * SL, k_hi, lds_base + B_BASE + (t % SB) * Col::BYTES,
             wave);
  };
  auto fetch_row = [&](int t) { row.fetch(k_lo + min(t, nk - 1) * SL, k_hi); };
  auto fetch_col = [&](int t) { col.fetch(k_lo + min(t, nk - 1) * SL, k_hi); };
  auto load_rows = [&](int t) {
    fetch_row(t);
#pragma unroll
    for (int q = 0; q < Row::Q; ++q) load_row(t, q);
  };
  auto load_cols = [&](int t) {
#pragma unroll
    for (int q = 0; q < Col::Q; ++q) load_col(t, q);
  };

  uint32_t ro[FM], co[FN];
#pragma unroll
  for (int x = 0; x < FM; ++x) ro[x] = RowR::lane_off(wm * TM + x * 32, lane);
#pragma unroll
  for (int y = 0; y < FN; ++y) co[y] = ColR::lane_off(wn * TN + y * 32, lane);
  f32x16 acc[FM][FN];
#pragma unroll
  for (int x = 0; x < FM; ++x)
#pragma unroll
    for (int y = 0; y < FN; ++y)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[x][y][r] = 0.f;
  bf16x8 fr[2][FM], fc[2][FN];
  // Fragment f of 16 k of slice t, in the order in which the MFMAs need them:
  // row 0, every column, the other rows.
  auto read = [&](int t, int kk, int f) {
    if (f >= 1 && f <= FN)
      fc[kk & 1][f - 1] =
          ColR::read(lds0 + B_BASE + (t % SB) * Col::BYTES, co[f - 1], kk, lane);
    else
      fr[kk & 1][f ? f - FN : 0] = RowR::read(lds0 + (t % SA) * Row::BYTES, ro[f ? f - FN : 0], kk, lane);
  };
  // The MFMAs of 16 k, in this order with the reads of the next 16 k (slice tr)
  // behind the first of them and `requests` requests of the ring between them:
  // a run of requests, from four waves at once, holds up the MFMAs behind it.
  auto step = [&](int kk, int tr, int requests, auto request) {
#pragma unroll
    for (int i = 0; i < NMF; ++i) {
      const int x = i / FN, y = i % FN;
      acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fc[kk & 1][y], fr[kk & 1][x], acc[x][y],
                                                         0, 0, 0);
      constexpr int NF = FM + FN, PER = (NF + NMF - 1) / NMF;
#pragma unroll
      for (int f = i * PER; f < (i + 1) * PER && f < NF; ++f) read(tr, (kk + 1) % KK, f);
#pragma unroll
      for (int q = 0; q < requests; ++q)
        if ((2 * q + 1) * NMF / (2 * requests) == i) request(q);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Before the last 16 k of slice t are multiplied, every wave has its
  // fragments of slice t in registers and waits for its loads of slice t + 1;
  // behind the barrier row slice t + SA and, under the next slice's first
  // MFMAs, column slice t + SB are requested into the stages of slice t, and
  // slice t + 1's first fragments are read under the last MFMAs, so no LDS
  // latency shows at the slice boundary.  Row slice t + 1 and column slice t + 1 come before row
  // slices t + 2 .. t + SA - 1 and column slices t + 2 .. t + SB - 1 in the
  // order of requests; only those may still be outstanding at the wait.
#pragma unroll
  for (int t = 0; t < SB - 1; ++t) {
    fetch_col(t);
    if (t < SA - 1) load_rows(t);
    load_cols(t);
  }
  fetch_col(SB - 1);
  load_rows(SA - 1);
  wait_vmcnt<(SA - 1) * Row::Q + (SB - 2) * Col::Q>();
  wg_barrier();
#pragma unroll
  for (int f = 0; f < FM + FN; ++f) read(0, 0, f);
  constexpr int CQ = (Col::Q + KK - 2) / (KK - 1);  // column requests of one step
  for (int t = 0; t < nk; ++t) {
#pragma unroll
    for (int kk = 0; kk + 1 < KK; ++kk)
      step(kk, t, max(0, min(CQ, Col::Q - kk * CQ)),
           [&](int q) { load_col(t + SB - 1, kk * CQ + q); });
    wait_vmcnt<(SA - 2) * Row::Q + (SB - 2) * Col::Q>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    fetch_col(t + SB);
    fetch_row(t + SA);
    step(KK - 1, t + 1, Row::Q, [&](int q) { load_row(t + SA, q); });
  }
  wait_vmcnt<0>();  // no load may land after the workgroup ends

  // The tile leaves through the ring's LDS in fp32, XC row fragments of every
  // wave at a time, so that rows are stored whole, 16 bytes per lane.  (Stored
  // from the MFMA layout, 8 bytes per lane in 32 rows at once, the output took
  // 12 to 22 us of a 52 to 64 us product, for 4 to 8 us of traffic.)
  typedef Staging<BM, BN, LDS> St;
  constexpr int XC = St::XC, ROWS = WM * XC * 32, PITCH = St::PITCH;  // PITCH in floats
  constexpr int CC = NC / V;
  constexpr int ITER = ROWS * CC / (W * MOE_WAVE);
  static_assert(ROWS * CC % (W * MOE_WAVE) == 0, "whole rounds");
  constexpr int U = ITER % 4 == 0 ? 4 : ITER % 3 == 0 ? 3 : ITER % 2 == 0 ? 2 : 1;
  typedef __attribute__((address_space(3))) f32x4 lds_f4;
  typedef __attribute__((address_space(3))) float lds_f;
  lds_f* out = (lds_f*)(smem);
  const int half = lane >> 5;
#pragma unroll
  for (int xc = 0; xc < FM; xc += XC) {
    __syncthreads();  // the ring, or the previous rows, are read
#pragma unroll
    for (int x = xc; x < xc + XC; ++x) {
      lds_f* o = out + ((wm * XC + x - xc) * 32 + (lane & 31)) * PITCH;
#pragma unroll
      for (int y = 0; y < FN; ++y)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          // GLU: accumulators 8 .. 15 are the up halves of columns 0 .. 15
          const int c = GLU ? (q >= 2 ? NC : 0) + (wn * TN + y * 32) / 2 + 8 * (q & 1)
                            : wn * TN + y * 32 + 8 * q;
          *(lds_f4*)(o + c + 4 * half) = f32x4{acc[x][y][4 * q], acc[x][y][4 * q + 1],
                                               acc[x][y][4 * q + 2], acc[x][y][4 * q + 3]};
        }
    }
    __syncthreads();
    // U chunks of 16 bytes of output per thread at once: one wave per SIMD has
    // nothing else to cover the LDS reads with
    for (int i0 = threadIdx.x; i0 < ROWS * CC; i0 += U * W * MOE_WAVE) {
      float g[U][V], u[U][V];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k * W * MOE_WAVE;
        const lds_f* o = out + i / CC * PITCH + i % CC * V;
#pragma unroll
        for (int j = 0; j < V; j += 4) {
          const f32x4 v = *(lds_f4*)(o + j);
#pragma unroll
          for (int c = 0; c < 4; ++c) g[k][j + c] = v[c];
          if constexpr (GLU) {
            const f32x4 w = *(lds_f4*)(o + NC + j);
#pragma unroll
            for (int c = 0; c < 4; ++c) u[k][j + c] = w[c];
          }
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k * W * MOE_WAVE, r = i / CC;
        out_chunk(r / (XC * 32) * TM + xc * 32 + r % (XC * 32), i % CC * V, g[k], u[k]);
      }
    }
  }
}

// Workgroup `block` of a product; smem: the ring.
template <bool RS, bool CS, int BM, int BN, bool GLU, bool PART>
__device__ __forceinline__ void mma_tile(const Mma& a, int block, unsigned char* smem) {
  static_assert(!GLU || (!CS && !PART), "pairs of gate and up rows: y = x w^T only");
  int mt, nt, split;
  if (!tile_of(a, block, mt, nt, split)) return;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
  constexpr int NC = GLU ? BN / 2 : BN;  // output columns of the tile
  const int m0 = mt * BM, n0 = nt * NC;
  const int k_lo = split * a.per_split, k_hi = min(a.K, k_lo + a.per_split);
  Operand<RS, false, BM, W> row;
  Operand<CS, GLU, BN, W> col;
  row.init(a.r + (RS ? m0 : m0 * a.ldr), a.ldr, min(BM, a.M - m0), wave, lane);
  col.init(a.c + (CS ? n0 : n0 * a.ldc), a.ldc, min(NC, a.N - n0), wave, lane,
           GLU ? a.N * a.ldc : 0);
  mma_core<RS, CS, BM, BN, GLU, PART ? 4 : 8>(
      row, col, k_lo, k_hi, smem, [&](int r, int c, float* g, float* u) {
        const int m = m0 + r, n = n0 + c;
        if (m >= a.M || n >= a.N) return;
        if constexpr (PART)
          store4(a.part + (static_cast<size_t>(split) * a.M + m) * a.N + n, g);
        else
          finish<uint16_t, GLU, 8>(a.e, m, n, a.N, g, u);
      });
}

template <bool RS, bool CS, int BM, int BN, int WGS, bool GLU, bool PART>
__global__ __launch_bounds__(W* MOE_WAVE) __attribute__((amdgpu_waves_per_eu(WGS, WGS)))
void mma_kernel(Mma a) {
  extern __shared__ __align__(16) unsigned char smem[];
  mma_tile<RS, CS, BM, BN, GLU, PART>(a, blockIdx.x, smem);
}

// Both products of a small backward pass and the bias gradient's last sum in
// one launch: workgroups from dw0 on are dw's, from bias0 on the bias's.  Each
// alone leaves most CUs empty or waits for memory.
template <bool PX, bool PW>
__global__ __launch_bounds__(W* MOE_WAVE) __attribute__((amdgpu_waves_per_eu(2, 2)))
void mma_pair_kernel(Mma dx, Mma dw, BiasSum b, int dw0, int bias0) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int block = blockIdx.x;
  if (block < dw0) mma_tile<false, true, 128, 128, false, PX>(dx, block, smem);
  else if (block < bias0) mma_tile<true, true, 128, 128, false, PW>(dw, block - dw0, smem);
  else bias_sum<uint16_t>(b, block - bias0, reinterpret_cast<float*>(smem));
}

}  // namespace lin
}  // namespace moe
