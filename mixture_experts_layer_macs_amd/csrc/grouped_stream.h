// bf16 gradients of many experts, one workgroup per CU that stays and walks its
// tiles of 256 x 256, the ring of linear_mma.h running on across their borders:
//
//   DW  dW_e = sum over e's rows of dz_r x_r^T
//   DX  dx_r = dz_r W_e
//
// An expert's reductions are short (DW: 8 slices of 64 rows at 512 rows), so a tile
// is half start and output.  Here a tile's first two slices are requested under the
// last two of the tile before it, and the output leaves through the one ring stage
// that is free then (32 KB, 64 rows at a time, already bf16); its stores go out
// behind those requests, and the wait of the next tile's first slice lets them be
// outstanding.  Loads and stores share one in-order counter, so every wave issues
// the same number of stores, those outside the matrix at an offset that the
// buffer's bounds drop.
//
// DX: an expert's rows are cut into units of 64 and these shared out evenly over its
// tiles; the waves hold them in fragments of 32 in turn, so that a tile of fewer
// than four units leaves out the MFMAs of whole fragments in every wave alike.
//
// Measured, DX of the spread tokens below: 511 us, a workgroup per tile 583.
// DW, 128 experts of 1536 x 2048: 512 rows each 470 us (0.88 PFLOP/s; a
// workgroup per tile 530, the library's batched product 600), 64 rows each 200 (250;
// 805 MB written, 118 at the rate of a fill); 8192 tokens as a router spreads them
// (up to 3700 rows) 541 to 567 (656).
#pragma once

#include <type_traits>

#include "grouped_common.h"
#include "grouped_mma.h"
#include "grouped_plan.h"

namespace moe {
namespace grp {

constexpr int ST = 256;                       // tile edge
constexpr int ST_STAGE = ST * SLICE * 2;      // bytes of a ring stage
constexpr int ST_LDS = (SA + SB) * ST_STAGE;  // 160 KB

// Who works on what, made on the device by a workgroup of the launch before: the
// experts in descending order of their rows, dealt to the 8 XCDs there and back
// (0 .. 7, 7 .. 0, ..), so that an expert's operands stay in one L2 and, of experts
// of like popularity, each XCD gets about an eighth of the rows.  An XCD's
// workgroups draw its tiles by tickets, the large experts' first.  (Tiles of a list
// in the experts' order dealt out in turns: 640 us for the 567 above; all workgroups
// drawing from one list: 599.)  An expert is not cut, and no XCD takes another's
// tiles, so the fullest one decides.  By the deal alone it has, times the mean of 128
// experts: 1.04 to 1.3 with the spread above, 1.29 with four experts ahead by 2 in
// the logits, 1.43 by Zipf's law with 1.1, 2 where only four have rows and 8 where
// only one has (whole backward passes of 65536 rows, us: 1081, 1147, 1233, 1910, 5739;
// even groups 1004).
struct alignas(16) PlanEntry {
  int32_t e, lo, hi, none;
};
struct Plan {
  PlanEntry entry[8][MOE_WAVE];  // e < 0: none
  int32_t ticket[2][8];          // tiles drawn, of DX and of DW
};
static_assert(STREAM_EXPERTS == 8 * MOE_WAVE, "an entry for each lane");

// A workgroup of 256 threads.
__device__ __forceinline__ void make_plan(const Groups& g, Plan* plan) {
  __shared__ int rows[STREAM_EXPERTS];
  for (int i = threadIdx.x; i < STREAM_EXPERTS; i += 256) {
    (&plan->entry[0][0])[i] = PlanEntry{-1, 0, 0, 0};
    if (i < g.N) {
      const Span s = span_of(g, i);
      rows[i] = s.hi - s.lo;
    }
  }
  if (threadIdx.x < 16) (&plan->ticket[0][0])[threadIdx.x] = 0;
  __syncthreads();  // also between the two writers of an entry
  for (int i = threadIdx.x; i < g.N; i += 256) {
    const int mine = rows[i];
    int rank = 0;
    for (int j = 0; j < g.N; ++j) rank += rows[j] > mine || (rows[j] == mine && j < i);
    const int xcd = rank / 8 % 2 ? 7 - rank % 8 : rank % 8;
    const Span s = span_of(g, i);
    plan->entry[xcd][rank / 8] = PlanEntry{i, s.lo, s.hi, 0};
  }
}

struct StreamTile {
  int e, lo, len;  // expert, first row of its reduction (DX: of the tile), reduction
  int m0, rows;    // first output row, rows
  int n0, width;   // first column, columns
  int live;        // units of 64 rows
};

// The row tiles of an expert: `first` of height + 1 units, then the others of height.
struct Cut {
  int tiles, height, first;
};
__device__ __forceinline__ Cut cut_of(int rows) {
  const int units = (rows + UNIT - 1) / UNIT, tiles = (units + 3) / 4;
  const int height = tiles ? units / tiles : 0;
  return {tiles, height, units - height * tiles};
}

// The tiles of the workgroup's XCD, an entry of the plan in each lane.
template <int MODE>
struct StreamTiles {
  const Prod& p;
  int tm, tn, e, lo, hi, incl, end;

  __device__ __forceinline__ StreamTiles(const Prod& q, const Plan* plan) : p(q) {
    tm = (p.W + ST - 1) / ST;  // DW
    tn = (p.K + ST - 1) / ST;
    const PlanEntry own = plan->entry[blockIdx.x % 8][lane_id()];
    e = own.e;
    lo = own.lo;
    hi = own.hi;
    incl = wave_incl_scan(e < 0 ? 0 : (MODE == DW ? tm : cut_of(hi - lo).tiles) * tn);
    end = read_lane(incl, MOE_WAVE - 1);
  }
  __device__ __forceinline__ StreamTile tile(int i) const {  // i < end
    const int l = __builtin_ctzll(__ballot(incl > i));
    const int first = read_lane(lo, l), count = read_lane(hi, l) - first;
    const Cut c = cut_of(count);
    const int height = MODE == DW ? tm : c.tiles;
    int mt, nt;
    banded(i - (read_lane(incl, l) - height * tn), height, tn, mt, nt);
    StreamTile t;
    t.e = read_lane(e, l);
    if (MODE == DW) {
      t.lo = first;
      t.len = count;
      t.m0 = uniform(mt * ST);
      t.rows = uniform(min(ST, p.W - t.m0));
      t.live = 4;
    } else {
      t.live = uniform(c.height + (mt < c.first));
      t.m0 = t.lo = uniform(first + (mt * c.height + min(mt, c.first)) * UNIT);
      t.rows = uniform(min(t.live * UNIT, first + count - t.m0));
      t.len = p.W;
    }
    t.n0 = uniform(nt * ST);
    t.width = uniform(min(ST, p.K - t.n0));
    return t;
  }
};

// Barrier that leaves loads and stores outstanding.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

template <int MODE>
__device__ __forceinline__ void stream_product(const Prod& p, Plan* plan, unsigned char* smem) {
  constexpr bool RS = MODE == DW;
  typedef Operand<RS, false, ST, lin::W> Row;
  typedef Operand<true, false, ST, lin::W> Col;
  typedef Reader<RS, ST> RowR;
  typedef Reader<true, ST> ColR;
  constexpr int FM = 4, FN = 4, KK = SLICE / 16, Q = 8, BASE = SA * ST_STAGE;
  constexpr int STORES = 32;  // of a whole tile, per wave
  static_assert(Row::Q == Q && Col::Q == Q && WM == 2 && WN == 2 && SA == 2 && SB == 3, "the waits' counts");
  typedef __attribute__((address_space(3))) unsigned char lds_byte;
  typedef __attribute__((address_space(3))) int32_t lds_int;
  typedef __attribute__((address_space(3))) u32x2 lds_u2;
  typedef __attribute__((address_space(3))) lin::u32x4 lds_u4;

  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
  const int wm = wave / WN, wn = wave % WN;
  const StreamTiles<MODE> tiles(p, plan);
  // The first tile goes by the workgroup's number, the others by ticket: drawn by
  // one thread, handed round through LDS that is free at the time.
  auto draw = [&]() __attribute__((always_inline)) {
    return threadIdx.x == 0
               ? static_cast<int32_t>(gridDim.x / 8) + atomicAdd(&plan->ticket[MODE == DW][blockIdx.x % 8], 1)
               : 0;
  };
  auto hand_round = [&](lds_byte* s, int32_t drawn) __attribute__((always_inline)) {
    if (threadIdx.x == 0) *(lds_int*)s = drawn;
    lds_barrier();
    const int v = uniform(*(lds_int*)s);
    lds_barrier();
    return min(v, tiles.end);
  };

  // ------------------------------------------------------------- the requests
  // The tile that is multiplied, that of the next request with its slice, and the
  // one after that if it is drawn already (-1: not).  Experts without rows come
  // last: the first tile without a reduction ends the product.
  int here = blockIdx.x / 8, ahead = here, next = -1, slice = 0, slices = 0, kend = 1;
  int queue[2] = {-1, -1};  // tiles requested behind `here`, in order
  bool more = false;
  if (here >= tiles.end) return;
  Row row;
  Col col;
  auto aim = [&]() __attribute__((always_inline)) {
    slice = 0;
    StreamTile t;
    t.len = 0;
    if (ahead < tiles.end) t = tiles.tile(ahead);
    more = t.len > 0;
    // otherwise one k of the last tile again and again, into stages that are not read
    kend = more ? t.len : 1;
    if (!more) return;
    slices = (t.len + SLICE - 1) / SLICE;
    const uint16_t *r = static_cast<const uint16_t*>(p.r), *c = static_cast<const uint16_t*>(p.c);
    row.init(r + static_cast<size_t>(t.lo) * p.W + (RS ? t.m0 : 0), p.W, t.rows, wave, lane);
    col.init(c + (RS ? static_cast<size_t>(t.lo) : static_cast<size_t>(t.e) * p.W) * p.K + t.n0, p.K, t.width,
             wave, lane);
  };
  // free: the stage that this slice's columns are about to take
  auto begin = [&](int free) __attribute__((always_inline)) {
    if (more && slice == slices) {
      if (next < 0) next = hand_round((lds_byte*)(smem + BASE + free * ST_STAGE), draw());
      ahead = next;
      next = -1;
      queue[queue[0] < 0 ? 0 : 1] = ahead;
      aim();
    }
    row.fetch(slice * SLICE, kend);
    col.fetch(slice * SLICE, kend);
  };
  const uint32_t lds_base = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((lds_byte*)(smem))));
  lds_cbyte* lds0 = (lds_cbyte*)(smem);
  auto load_row = [&](int q, int stage) {
    row.load(q, slice * SLICE, kend, lds_base + stage * ST_STAGE, wave);
  };
  auto load_col = [&](int q, int stage) {
    col.load(q, slice * SLICE, kend, lds_base + BASE + stage * ST_STAGE, wave);
  };

  // ------------------------------------------------------------- the product
  int rs = 0, cs = 0;   // stages of the slice that is multiplied
  bool stored = false;  // the output's stores lie between the last requests
  uint32_t ro[FM], co[FN];
#pragma unroll
  for (int x = 0; x < FM; ++x) ro[x] = RowR::lane_off(x * UNIT + wm * 32, lane);
#pragma unroll
  for (int y = 0; y < FN; ++y) co[y] = ColR::lane_off(wn * (ST / 2) + y * 32, lane);
  f32x16 acc[FM][FN];
  bf16x8 fr[2][FM], fc[2][FN];
  auto clear = [&](int x) {
#pragma unroll
    for (int y = 0; y < FN; ++y)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[x][y][i] = 0.f;
  };
  auto read = [&](int r, int c, int kk, int f) {
    if (f >= 1 && f <= FN)
      fc[kk & 1][f - 1] = ColR::read(lds0 + BASE + c * ST_STAGE, co[f - 1], kk, lane);
    else
      fr[kk & 1][f ? f - FN : 0] = RowR::read(lds0 + r * ST_STAGE, ro[f ? f - FN : 0], kk, lane);
  };
  // As in mma_core: the MFMAs of 16 k, the reads of the next 16 k from stages r and
  // c behind the first, the requests between them; live: row fragments of a wave.
  auto step = [&](auto live, int kk, int r, int c, int requests, auto request)
      __attribute__((always_inline)) {
    constexpr int LIVE = decltype(live)::value;
#pragma unroll
    for (int i = 0; i < FM * FN; ++i) {
      const int x = i / FN, y = i % FN;
      if (x < LIVE)
        acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fc[kk & 1][y], fr[kk & 1][x],
                                                             acc[x][y], 0, 0, 0);
      if (i < FM + FN) read(r, c, (kk + 1) % KK, i);
#pragma unroll
      for (int q = 0; q < requests; ++q)
        if ((2 * q + 1) * FM * FN / (2 * requests) == i) request(q);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // Slice g, while column slice g + 2 and, behind the barrier, row slice g + 2 are
  // requested.  The wait is for row and column slice g + 1; behind those come, in
  // this order, the stores of an output in between and column slice g + 2.
  auto one_slice = [&](auto live) __attribute__((always_inline)) {
    const int rn = rs ^ 1, cn = cs == 2 ? 0 : cs + 1, cr = cs == 0 ? 2 : cs - 1;
    begin(cr);
    step(live, 0, rs, cs, 3, [&](int q) { load_col(q, cr); });
    step(live, 1, rs, cs, 3, [&](int q) { load_col(3 + q, cr); });
    step(live, 2, rs, cs, 2, [&](int q) { load_col(6 + q, cr); });
    if (stored) wait_vmcnt<STORES + Q>();
    else wait_vmcnt<Q>();
    stored = false;
    lds_barrier();
    step(live, 3, rn, cn, Q, [&](int q) { load_row(q, rs); });
    slice += more;
    rs = rn;
    cs = cn;
  };

  // -------------------------------------------------------------- the output
  auto output = [&](const StreamTile& t) __attribute__((always_inline)) {
    constexpr int CH = ST / 8;  // 16-byte chunks of a row
    // the stage of the slice behind us: its next request is still to come
    lds_byte* s = (lds_byte*)(smem + BASE + (cs == 0 ? 2 : cs - 1) * ST_STAGE);
    int32_t drawn = 0;
    const bool drawing = next < 0 && more;
    if (drawing) drawn = draw();
    const uint32_t bytes = static_cast<uint32_t>(p.K) * 2;
    const auto rsrc = store_rsrc(
        static_cast<uint16_t*>(p.e.y) +
            ((RS ? static_cast<size_t>(t.e) * p.W : 0) + t.m0) * p.K + t.n0,
        (t.rows - 1) * bytes + t.width * 2);
    // The lane's places are worked out anew for each output: held over the product
    // they would take the registers of a third of the fragments.
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int half = tid / 32 % 2, wr = tid % 32, ch = tid % CH, r0 = tid / CH;
#pragma unroll
    for (int x = 0; x < FM; ++x) {
      if (x >= t.live) {
        clear(x);
        continue;
      }
#pragma unroll
      for (int y = 0; y < FN; ++y)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16& a = acc[x][y];
          const int c = wn * (CH / 2) + y * 4 + q;
          *(lds_u2*)(s + (wm * 32 + wr) * (ST * 2) + ((c ^ wr) << 4) + 8 * half) =
              u32x2{pack2(a[4 * q], a[4 * q + 1]), pack2(a[4 * q + 2], a[4 * q + 3])};
        }
      clear(x);
      lds_barrier();
      lin::u32x4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = r0 + 8 * j;
        v[j] = *(lds_u4*)(s + r * (ST * 2) + ((ch ^ (r & 31)) << 4));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int m = x * UNIT + r0 + 8 * j;
        buf_store16(rsrc, ch * 8 < t.width ? m * bytes + ch * 16 : OOB_OFF, v[j]);
      }
      lds_barrier();
    }
    stored = t.live == 4;
    if (drawing) next = hand_round(s, drawn);
  };

  aim();
  if (more) {  // the first tile has a reduction
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      begin(2);
#pragma unroll
      for (int q = 0; q < Q; ++q) load_row(q, g);
#pragma unroll
      for (int q = 0; q < Q; ++q) load_col(q, g);
      slice += more;
    }
    wait_vmcnt<2 * Q>();
    wg_barrier();
#pragma unroll
    for (int f = 0; f < FM + FN; ++f) read(0, 0, 0, f);
#pragma unroll
    for (int x = 0; x < FM; ++x) clear(x);
    while (here < tiles.end) {
      const StreamTile t = tiles.tile(here);
      if (t.len == 0) break;
      auto multiply = [&](auto live) __attribute__((always_inline)) {
        for (int k = 0; k < t.len; k += SLICE) one_slice(live);
      };
      if (MODE == DW || t.live == 4) multiply(std::integral_constant<int, 4>());
      else if (t.live == 3) multiply(std::integral_constant<int, 3>());
      else if (t.live == 2) multiply(std::integral_constant<int, 2>());
      else multiply(std::integral_constant<int, 1>());
      output(t);
      here = queue[0];
      queue[0] = queue[1];
      queue[1] = -1;
    }
  }
  wait_vmcnt<0>();  // no load may land after the workgroup ends
  // DW: what is left are weights of experts without rows: zeros.
  while (MODE == DW && here < tiles.end) {
    const StreamTile t = tiles.tile(here);
    uint16_t* out =
        static_cast<uint16_t*>(p.e.y) + (static_cast<size_t>(t.e) * p.W + t.m0) * p.K + t.n0;
    for (int j = threadIdx.x; j < t.rows * (ST / 8); j += lin::W * MOE_WAVE) {
      const int r = j / (ST / 8), c = j % (ST / 8) * 8;
      if (c < t.width)
        *reinterpret_cast<lin::u32x4*>(out + static_cast<size_t>(r) * p.K + c) = lin::u32x4{0, 0, 0, 0};
    }
    lds_barrier();
    here = hand_round((lds_byte*)smem, draw());
  }
}

template <int MODE>
__global__ __launch_bounds__(lin::W* MOE_WAVE) __attribute__((amdgpu_waves_per_eu(1, 1)))
void grouped_stream_mma_kernel(Prod p, Plan* plan) {
  extern __shared__ __align__(16) unsigned char smem[];
  stream_product<MODE>(p, plan, smem);
}

}  // namespace grp
}  // namespace moe
