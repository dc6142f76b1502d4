// window_bwd_sm100.cuh -- gradients of attention over a sliding window with sink tokens and
// grouped key/value heads (sm_100a).
//
//   P = exp(scale Q K^T - lse) (unseen entries 0),  dS = P o (dO V^T - D),  D = rowsum(dO o O)
//   dQ = scale dS K,   dV = sum over the group's heads of P^T dO,   dK = scale sum of dS^T Q
//
// Two launches of one kernel, so that no sum needs atomics (results do not depend on the run,
// and there is no fp32 accumulator in memory): one holds a tile of queries and streams the keys
// that it sees, for dQ (and D, which it writes for the other); one holds a tile of keys and
// streams the queries of all the group's heads that see it, for dK and dV.  That recomputes two
// of seven products; adding up dQ over the key tiles instead would move 32 KB through L2
// reductions for every 64 x 128 tile, 1.2 GB at 4096 tokens of 2 x 32 heads.
//
// In both, a unit keeps a pair of 128-row tiles X1, X2 (Q, dO | K, V) in shared memory and walks
// over pairs of 128-row tiles Y1, Y2 (K, V | Q, dO) through a ring.  Per step, on the tensor cores:
//   S = X1 Y1^T,  T = X2 Y2^T      (lane = row of X, column = row of Y; fp32 in TMEM)
//   elementwise: P = 2^(scale_log2 S - lse_log2), dS = P (T - D), packed to 16 bits over S and T
//   dQ += dS Y1   |   dV += P Y2,  dK += dS Y1     (A from TMEM, B the tiles read MN-major)
// in the order  dV(i)  S(i + 1)  dK(i)  T(i + 1): the exponentials of step i + 1 run while the
// tensor cores do dK(i) and T(i + 1), its dS while they do dV(i + 1) and S(i + 2), so one S and
// one T (256 TMEM columns; the gradients take the rest) keep both sides busy.  The queries'
// launch has no dV; there S(i + 1) and T(i + 1) (T has two buffers) follow as soon as S(i) has
// been read, before dQ(i): the chain T, dS, dQ, T of one buffer took 280 us where this took 272.
//
// Roundings: P and dS of the keys' launch are rounded once to the inputs' type, which leaves dV and
// dK 1.4 times the error of a product in fp32 that is rounded at its end.  dQ would be at 1.5 to 1.6
// times, so there dS enters as the sum of two 16-bit values (the second is what the first was
// rounded by, in the half of T's columns that the first leaves free), a product each: 272 -> 327 us.
//
// Range: dS carries the size of dO and of V, and fp16 has 2^-24 to 2^16 (dO of 1e-3 left dQ and dK at 3
// times their own rounding, dO V^T past 65504 gave NaN).  So in fp16 dS enters as 2^e dS, with e from a
// bound of |T - D|, |dO| |v| + |D| (and P <= 1), that puts it below 2^14, and the gradient is taken back by
// 2^-e: dQ's e is its row's, from |dO| of the row and the largest |v| among the unit's keys; dK's is the
// unit's, from the largest |dO| and |D| of its queries, by 128 of them, which the queries' launch leaves
// behind.  Typical products lie 2^4 to 2^8 below the bound, so P down to 2^-17 and rows of 2^-10 of the
// largest still enter as normal numbers.  P enters dV as 2^12 P.  The powers of two ride in the exponent
// of P and in the subtraction of D; what they cost is the bounds (a small launch over V, and some 0.5 us a
// unit): 4096 tokens in fp16 641 -> 664 us, 1000 tokens 37.1 -> 40.5.  bf16 has fp32's range and none of it.
//
// What bounds it, at 4096 tokens of 2 x 32 heads over 8, 128 channels, window 1024, bf16: the queries'
// launch takes 331 us, the keys' 316, the join 5; the tensor cores work 40 and 47 % of that, the
// issue slots 36 and 29 %, DRAM 11 %.  A unit is 9 or 10 steps and about 5 us of them its start and
// end (X1 and X2 have one buffer: two do not fit beside the ring at 128 channels; at 64 they would),
// in which the tensor cores wait.
//
// Roles (576 threads): warps 0-15 elementwise and epilogue (four per TMEM lane quarter, 32 of the
// 128 columns each), warp 16 producer, warp 17 MMA issuer.  Units are claimed with cluster launch
// control, as in prefill_sm100.cuh.
// (With 64-row Y tiles and S and T double-buffered, both launches took 690 us where 128-row tiles
// took 628: an M = 128, N = 64 product of two shared-memory operands costs as
// much as one with N = 128.)
//
// TMEM columns: S [0, 128) (P packed over it), T [128, 256) (dS; the queries' second one is
// [384, 512)), gradients at 256 and, dK, 384.
#pragma once

#include "window_fwd_sm100.cuh"

namespace attn_b200 {

struct WindowBwdParams {
  CUtensorMap tm_x1, tm_x2;  // resident tiles: 128 rows (queries: pack heads x 128 / pack positions)
  CUtensorMap tm_y1, tm_y2;  // streamed tiles: box (64, 1, 128, 1), 128B swizzle
  CUtensorMap tm_y1_8, tm_y2_8;  // the queries' launch: the same in boxes of 8 rows
  const void* o;             // the queries' launch: O, for D; elements from batch to batch, query to
  long long o_batch, o_query, o_head;  // query, head to head
  const float* lse;          // [B, H, Nq]
  float* dsum;               // [B, H, Nq]: D, written by the queries' launch
  void* g1;                  // dQ | dV
  void* g2;                  // - | dK
  float* part;               // the keys' launch: [parts][2][128][D] of split units
  const float* vmax;         // fp16: [B, Hkv, ceil(Nk / 128)]: largest |v|^2 of 128 keys, and
  unsigned* qmax;            // [B, Hkv, ceil(Nq / 128)][2]: largest |dO| (a bound of it) and |D| of 128
                             // queries, as bits of floats that are not negative
  int* status;
  int B, H, Hkv, Nq, Nk;
  int lg_pack;               // the queries' launch
  int window, sinks;
  int n_xtiles;              // X tiles along the sequence
  int sink_tiles;            // keys: tiles with sinks come first, their queries split over
  int sink_splits, splits;   // sink_splits units; the others' over splits
  float scale, scale_log2;
  unsigned long long timeout_ns;
  int inject;                // test hook: 1 = the first tile X1 never counts as landed
};

template <int D>
struct WindowBwdCfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kBox = 128 * 128;                     // 128 rows x 64 elements x 2 bytes
  static constexpr int kTile = kBoxes * kBox;
  static constexpr int kSlots = D == 128 ? 5 : 8;            // of the ring: Y1, Y2 tiles in turn
  static constexpr int kOffY = 2 * kTile;                    // X1, X2, then the ring
  // keys: float [2][-lse, -D][128] of the steps' columns; queries: float [4][128], quarters of D
  static constexpr int kOffRow = kOffY + kSlots * kTile;
  static constexpr int kOffBar = kOffRow + 2048;
  static constexpr int kBarXFull = 0, kBarXEmpty = 2, kBarS = 4, kBarT = 5, kBarP = 7, kBarDS = 8, kBarAcc = 10,
                       kBarMmaDone = 11, kBarClc = 12, kBarUnitFull = 13, kBarUnitEmpty = 15, kBarYFull = 17,
                       kBarYEmpty = kBarYFull + kSlots, kBarMeet = kBarYEmpty + kSlots,
                       kNumBars = kBarMeet + 4;
  static constexpr int kUnitInts = 8;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;    // tmem slot, abort flag, unit slots
  static constexpr int kOffClc = (kOffMisc + 8 + 2 * kUnitInts * 4 + 15) / 16 * 16;
  static constexpr int kOffNorm = kOffClc + 16;              // queries, fp16: uint8 [4][128], quarters of |dO|^2
  static constexpr int kSmemBytes = kOffNorm + 512;          // the shared memory is declared 1 KB aligned
  static constexpr int kEwWarps = 16, kProducerWarp = 16, kMmaWarp = 17, kThreads = 576;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

struct WindowBwdUnit {
  int b, h;   // batch; first head of the tile | key/value head
  int x0;     // first query | key of the X tiles
  int a, c;   // queries' launch: sink8, shift (WindowUnit) | first query, 128-query tiles of a head
  int s0, n;  // first step and steps (n < 0: no more units)
  int part;   // keys: index of the partial gradients, -1: none
};

template <bool kKeys>
__device__ __forceinline__ WindowBwdUnit window_bwd_unit(const WindowBwdParams& p, int unit) {
  WindowBwdUnit u;
  const long long diag = (long long)p.Nk - p.Nq;
  if constexpr (kKeys) {
    const int heads = p.B * p.Hkv;
    const int sink_units = heads * p.sink_tiles * p.sink_splits;
    int rest = unit, splits, tiles, first_tile;
    if (unit < sink_units) {
      splits = p.sink_splits;
      tiles = p.sink_tiles;
      first_tile = 0;
      u.part = splits > 1 ? unit : -1;
    } else {
      rest = unit - sink_units;
      splits = p.splits;
      tiles = p.n_xtiles - p.sink_tiles;
      first_tile = p.sink_tiles;
      u.part = splits > 1 ? rest + (p.sink_splits > 1 ? sink_units : 0) : -1;
    }
    const int tile = rest / splits, sp = rest - tile * splits;
    const int bh = tile / tiles;
    u.b = bh / p.Hkv;
    u.h = bh - u.b * p.Hkv;
    u.x0 = 128 * (first_tile + tile - bh * tiles);
    const int last = min(u.x0 + 127, p.Nk - 1);
    // queries that see a key of the tile: [lo, hi)
    const long long lo = max(0LL, u.x0 - diag);
    const long long hi = u.x0 < p.sinks ? p.Nq : min((long long)p.Nq, last - diag + p.window);
    u.a = (int)min(lo, (long long)p.Nq);
    u.c = hi > lo ? (int)((hi - lo + 127) / 128) : 0;
    const long long steps = (long long)u.c * (p.H / p.Hkv);
    u.s0 = (int)(steps * sp / splits);
    u.n = (int)(steps * (sp + 1) / splits) - u.s0;
  } else {
    const int rows = 128 >> p.lg_pack, blocks = p.H >> p.lg_pack;
    const int bh = unit / p.n_xtiles;
    u.b = bh / blocks;
    u.h = (bh - u.b * blocks) << p.lg_pack;
    u.x0 = (unit - bh * p.n_xtiles) * rows;
    const long long pos = u.x0 + diag, hi = pos + min(rows, p.Nq - u.x0) - 1;
    int low = (int)max(0LL, pos - p.window + 1);
    u.a = (int)min(((long long)p.sinks + 7) / 8 * 8, 1LL << 30);
    if (u.a >= low) u.a = low = 0;
    u.c = low - u.a;
    u.s0 = 0;
    u.n = hi >= 0 ? (int)(hi - u.c) / 128 + 1 : 0;
    u.part = -1;
  }
  return u;
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_bits(uint32_t lo, uint32_t hi) {
  return f2_make(__uint_as_float(lo), __uint_as_float(hi));
}

// fp16: P of the keys' launch enters the products as 2^kPShift P, and dS as 2^e dS.
constexpr int kPShift = 12;
// e for |T - D| <= bound: 2^e bound lies in [2^13, 2^14).  (fp16 inputs: nonzero bounds lie in [2^-49, 2^42].)
__device__ __forceinline__ int ds_shift(float bound) {
  return min(max(13 - ((int)(__float_as_uint(bound) >> 23) - 127), -64), 64);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ float warp_max(float x) {  // of values that are not negative
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}

// fp16, before the queries' launch: the largest |v|^2 of each 128 keys of a head (a block each), and
// qmax set to 0.
template <int D>
__global__ void __launch_bounds__(256) attn_window_bwd_kernel_bounds(const void* v, float* vmax, unsigned* qmax, int Hkv,
                                                                     int Nk, int n_kblocks, long long n_qmax) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kLanes = D / 8, kPasses = 128 * kLanes / 256;  // lanes of a row; rows of a thread
  __shared__ unsigned top;
  if (threadIdx.x == 0) top = 0u;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n_qmax; i += gridDim.x * 256LL) qmax[i] = 0u;
  const int bh = blockIdx.x / n_kblocks, key0 = 128 * (blockIdx.x - bh * n_kblocks);
  const int b = bh / Hkv, hk = bh - b * Hkv;
  const int row = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
  uint4 x[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int key = key0 + row + i * (256 / kLanes);
    x[i] = key < Nk ? __ldg(static_cast<const uint4*>(v) + (((long long)b * Nk + key) * Hkv + hk) * kLanes + c)
                    : make_uint4(0u, 0u, 0u, 0u);
  }
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack2<false>(w[e]);
      s = fmaf(f.x, f.x, fmaf(f.y, f.y, s));
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    most = fmaxf(most, s);
  }
  most = warp_max(most);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) atomicMax(&top, __float_as_uint(most));
  __syncthreads();
  if (threadIdx.x == 0) vmax[blockIdx.x] = __uint_as_float(top);
}

template <int D, bool BF16, bool kKeys>
__global__ void __launch_bounds__(WindowBwdCfg<D>::kThreads, 1)
    attn_window_bwd_kernel(const __grid_constant__ WindowBwdParams p) {
  using C = WindowBwdCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + C::kOffBar;
  auto BAR = [&](int i) -> uint32_t { return bars + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  volatile int* unit_slot = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
  const uint32_t clc_resp = sbase + C::kOffClc;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx wctx{abort_flag, p.status, p.timeout_ns};
  const int G = p.H / p.Hkv;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the next launch may be set up

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(C::kBarXFull + i), p.inject == 1 && i == 0 ? 2 : 1);
      // queries: D is taken from dO (X2) by the elementwise warps
      mbar_init(BAR(C::kBarXEmpty + i), !kKeys && i == 1 ? 1 + C::kEwWarps : 1);
      mbar_init(BAR(C::kBarUnitFull + i), 1);
      mbar_init(BAR(C::kBarUnitEmpty + i), C::kEwWarps + 1);
    }
    mbar_init(BAR(C::kBarS), 1);
    mbar_init(BAR(C::kBarT), 1);
    mbar_init(BAR(C::kBarT + 1), 1);
    mbar_init(BAR(C::kBarP), C::kEwWarps);
    mbar_init(BAR(C::kBarDS), C::kEwWarps);
    mbar_init(BAR(C::kBarDS + 1), C::kEwWarps);
    mbar_init(BAR(C::kBarAcc), 1);
    // keys: the four warps of each part of the columns; queries: one for all warps
    for (int i = 0; i < 4; ++i) mbar_init(BAR(C::kBarMeet + i), kKeys ? 4 : C::kEwWarps);
    mbar_init(BAR(C::kBarMmaDone), 1);
    mbar_init(BAR(C::kBarClc), 1);
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(BAR(C::kBarYFull + s), 1);
      mbar_init(BAR(C::kBarYEmpty + s), 1);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  auto next_unit = [&](int k) -> WindowBwdUnit {
    mbar_wait_inline(BAR(C::kBarUnitFull + (k & 1)), (k >> 1) & 1, wctx);
    __syncwarp();
    const volatile int* us = unit_slot + (k & 1) * C::kUnitInts;
    WindowBwdUnit u;
    u.b = us[0];
    u.h = us[1];
    u.x0 = us[2];
    u.a = us[3];
    u.c = us[4];
    u.s0 = us[5];
    u.n = warp_flag(abort_flag) ? -1 : us[6];
    u.part = us[7];
    __syncwarp();
    if (lane == 0) mbar_arrive(BAR(C::kBarUnitEmpty + (k & 1)));
    return u;
  };

  // T of step g is there, or its dS.  The queries' T(g + 1) is issued before dS(g) is waited for,
  // so the elementwise warps can be a step ahead of the issuer: these barriers take turns there,
  // or a phase could end unseen.
  auto wait_step = [&](int bar, int g) {
    if constexpr (kKeys) mbar_wait_inline(BAR(bar), g & 1, wctx);
    else mbar_wait_inline(BAR(bar + (g & 1)), (g >> 1) & 1, wctx);
  };

  if (warp == C::kProducerWarp) {
    // ======================= producer: unit claims and loads =======================
    if (lane == 0) {
      tma_prefetch_map(&p.tm_x1);
      tma_prefetch_map(&p.tm_x2);
      tma_prefetch_map(&p.tm_y1);
      tma_prefetch_map(&p.tm_y2);
    }
    __syncwarp();
    int unit = blockIdx.x, nx = 0, nx_issued[2] = {0, 0}, g = 0, nclaim = 0;  // units with steps; X1, X2, ring items loaded
    for (int k = 0;; ++k) {
      WindowBwdUnit u{};
      if (unit >= 0) u = window_bwd_unit<kKeys>(p, unit);
      else u.n = -1;
      if (k >= 2) mbar_wait_inline(BAR(C::kBarUnitEmpty + (k & 1)), ((k >> 1) - 1) & 1, wctx);
      __syncwarp();
      if (lane == 0) {
        volatile int* us = unit_slot + (k & 1) * C::kUnitInts;
        us[0] = u.b;
        us[1] = u.h;
        us[2] = u.x0;
        us[3] = u.a;
        us[4] = u.c;
        us[5] = u.s0;
        us[6] = u.n;
        us[7] = u.part;
        mbar_arrive(BAR(C::kBarUnitFull + (k & 1)));
      }
      __syncwarp();
      if (unit < 0) break;
      if (!kKeys && u.n > 0) {
        // the rows of O that D is taken from, into L2 by the time the elementwise warps read them
        for (int r = lane; r < 128; r += 32) {
          const int query = u.x0 + (r >> p.lg_pack), head = u.h + (r & ((1 << p.lg_pack) - 1));
          if (query < p.Nq)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(__cvta_generic_to_global(
                             static_cast<const uint16_t*>(p.o) + u.b * p.o_batch + query * p.o_query + head * p.o_head)),
                         "r"(D * 2)
                         : "memory");
        }
        __syncwarp();
      }
      bool claimed = false;
      auto claim_next = [&]() {
        if (!claimed && !warp_flag(abort_flag)) {
          mbar_arrive_expect_tx_w(BAR(C::kBarClc), 16);
          clc_try_cancel_w(clc_resp, BAR(C::kBarClc));
          claimed = true;
        }
      };
      auto load_x = [&](int i) {
        if (nx > 0) mbar_wait_inline(BAR(C::kBarXEmpty + i), (nx - 1) & 1, wctx);
        __syncwarp();
        if (warp_flag(abort_flag)) return;
        mbar_arrive_expect_tx_w(BAR(C::kBarXFull + i), C::kTile);
        for (int bx = 0; bx < C::kBoxes; ++bx)
          tma_load_4d_w(sbase + i * C::kTile + bx * C::kBox, i ? &p.tm_x2 : &p.tm_x1, BAR(C::kBarXFull + i), bx * 64, u.h,
                        u.x0, u.b);
        ++nx_issued[i];
      };
      int head = 0, qt = 0;  // keys: head of the group and query tile of the step
      if (kKeys && u.n > 0) {
        head = u.s0 / u.c;
        qt = u.s0 - head * u.c;
      }
      for (int i = 0; i < u.n; ++i) {
        if (i == max(0, u.n - C::kSlots)) claim_next();
        int row, hd;
        bool mixed = false;
        if constexpr (kKeys) {
          row = u.a + 128 * qt;
          hd = u.h * G + head;
          if (++qt == u.c) {
            qt = 0;
            ++head;
          }
        } else {
          row = 128 * i + (128 * i >= u.a ? u.c : 0);
          hd = u.h / G;
          mixed = 128 * i < u.a && 128 * i + 128 > u.a;
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if (i == 0) load_x(y);
          const int st = g % C::kSlots;
          if (g >= C::kSlots) mbar_wait_inline(BAR(C::kBarYEmpty + st), (g / C::kSlots - 1) & 1, wctx);
          __syncwarp();
          if (warp_flag(abort_flag)) break;
          const uint32_t bar = BAR(C::kBarYFull + st), dst = sbase + C::kOffY + st * C::kTile;
          mbar_arrive_expect_tx_w(bar, C::kTile);
          if (!mixed) {
            for (int bx = 0; bx < C::kBoxes; ++bx)
              tma_load_4d_w(dst + bx * C::kBox, y ? &p.tm_y2 : &p.tm_y1, bar, bx * 64, hd, row, u.b);
          } else if (lane < 16) {
            // the tile in which the sinks end: lane l copies rows 8 l .. 8 l + 7
            const int key = row + 8 * lane + (row + 8 * lane >= u.a ? u.c : 0);
            for (int bx = 0; bx < C::kBoxes; ++bx)
              tma_load_4d(dst + bx * C::kBox + lane * 1024, y ? &p.tm_y2_8 : &p.tm_y1_8, bar, bx * 64, hd, key, u.b);
          }
          __syncwarp();
          ++g;
        }
        if (warp_flag(abort_flag)) break;
      }
      if (u.n > 0) ++nx;
      claim_next();
      int next = -1;
      if (claimed) {
        if (mbar_wait_inline(BAR(C::kBarClc), nclaim & 1, wctx)) next = clc_response_ctaid_x(clc_resp);
        else mbar_wait_drain_inline(BAR(C::kBarClc), nclaim & 1, p.timeout_ns);
        ++nclaim;
      }
      __syncwarp();
      unit = __shfl_sync(0xffffffffu, next, 0);
    }
    if (warp_flag(abort_flag)) {
      // let every copy this warp started land before the CTA can exit
      for (int i = 0; i < 2; ++i)
        if (nx_issued[i] > 0) mbar_wait_drain_inline(BAR(C::kBarXFull + i), (nx_issued[i] - 1) & 1, p.timeout_ns);
      for (int i = max(0, g - C::kSlots); i < g; ++i)
        mbar_wait_drain_inline(BAR(C::kBarYFull + i % C::kSlots), (i / C::kSlots) & 1, p.timeout_ns);
      __syncwarp();
    }
  } else if (warp == C::kMmaWarp) {
    // ======================= tcgen05 MMA issuer =======================
    constexpr uint32_t idesc_s = make_idesc_f16(128, 128, BF16, false, false);
    constexpr uint32_t idesc_g = make_idesc_f16(128, D, BF16, true, false);
    auto slot = [&](int item) -> uint32_t { return sbase + C::kOffY + (item % C::kSlots) * C::kTile; };
    // TMEM columns of T of step `step`
    auto t_col = [&](int step) -> uint32_t { return !kKeys && (step & 1) ? 384u : 128u; };
    // S (y = 0) or T (y = 1) of step `step`
    auto issue_st = [&](int y, int step) {
      const int item = 2 * step + y;
      mbar_wait_inline(BAR(C::kBarYFull + item % C::kSlots), (item / C::kSlots) & 1, wctx);
      __syncwarp();
      tc_fence_after_sync();
      if (warp_flag(abort_flag)) return;
      const uint64_t a = make_sdesc_sw128(sbase + y * C::kTile, 16, 1024), b = make_sdesc_sw128(slot(item), 16, 1024);
      const uint32_t d = tmem + (y ? t_col(step) : 0u);
      if constexpr (D == 128) mma_f16_ss_k128_w<C::kBox>(d, a, b, idesc_s, 0u);
      else mma_f16_ss_k64_w(d, a, b, idesc_s, 0u);
      tc_commit_w(BAR((y ? C::kBarT + (kKeys ? 0 : step & 1) : C::kBarS)));
      if (y && !kKeys) tc_commit_w(BAR(C::kBarYEmpty + item % C::kSlots));  // V is done with
    };
    // a gradient (columns at acc) += P or dS (columns at a) times ring item `item`: 128 rows
    auto issue_g = [&](uint32_t acc, uint32_t a, int item, bool accumulate) {
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)  // 16 rows of Y a k-step: 8 packed TMEM columns
        mma_f16_ts_w(tmem + acc, tmem + a + (kk >> 1) * 32 + (kk & 1) * 8,
                     make_sdesc_sw128(slot(item) + kk * 2048, C::kBox, 1024), idesc_g, accumulate || kk > 0 ? 1u : 0u);
    };
    auto release_x = [&](int y) {
      if (!warp_flag(abort_flag)) tc_commit_w(BAR(C::kBarXEmpty + y));
    };
    int g = 0, nx = 0;  // steps and units with steps so far
    for (int k = 0;; ++k) {
      const WindowBwdUnit u = next_unit(k);
      if (u.n < 0) break;
      if (u.n == 0) continue;
      for (int y = 0; y < 2; ++y) {
        mbar_wait_inline(BAR(C::kBarXFull + y), nx & 1, wctx);
        __syncwarp();
        issue_st(y, g);
        if (u.n == 1) release_x(y);
      }
      for (int i = 0; i < u.n; ++i, ++g) {
        mbar_wait_inline(BAR(C::kBarP), g & 1, wctx);
        __syncwarp();
        tc_fence_after_sync();
        if (kKeys && !warp_flag(abort_flag)) {
          issue_g(256, 0, 2 * g + 1, i > 0);
          tc_commit_w(BAR(C::kBarYEmpty + (2 * g + 1) % C::kSlots));
        }
        if (i + 1 < u.n) {
          issue_st(0, g + 1);
          if (i + 2 == u.n) release_x(0);
          if constexpr (!kKeys) {
            issue_st(1, g + 1);
            if (i + 2 == u.n) release_x(1);
          }
        }
        wait_step(C::kBarDS, g);
        __syncwarp();
        tc_fence_after_sync();
        if (!warp_flag(abort_flag)) {
          issue_g(kKeys ? 384 : 256, t_col(g), 2 * g, i > 0);
          if constexpr (!kKeys) issue_g(256, t_col(g) + 16, 2 * g, true);
          tc_commit_w(BAR(C::kBarYEmpty + (2 * g) % C::kSlots));
          if (i + 1 == u.n) tc_commit_w(BAR(C::kBarAcc));
        }
        if (kKeys && i + 1 < u.n) {
          issue_st(1, g + 1);
          if (i + 2 == u.n) release_x(1);
        }
      }
      ++nx;
    }
    // every MMA (and every commit arrive) has landed before TMEM is released
    tc_commit_w(BAR(C::kBarMmaDone));
    mbar_wait_drain_inline(BAR(C::kBarMmaDone), 0, p.timeout_ns);
    __syncwarp();
  } else {
    // ======================= elementwise warps 0-15 =======================
    const int part = warp >> 2;               // which 32 of a step's 128 columns
    const int r = (warp & 3) * 32 + lane;     // TMEM lane: row of the X tiles
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + part * 32;
    const long long diag = (long long)p.Nk - p.Nq;
    const float cs = p.scale_log2;
    float* rowbuf = reinterpret_cast<float*>(smem + C::kOffRow);
    // what the launch before wrote: keys: D; fp16: the bounds
    if constexpr (kKeys || !BF16) asm volatile("griddepcontrol.wait;" ::: "memory");
    int g = 0, nx = 0;  // steps and units with steps so far
    WindowBwdUnit u = next_unit(0);
    // Of the unit that u is: this lane's row of the X tiles, and what is loaded of it ahead, while
    // the unit before is finished (its first step waited 1 us for it otherwise).
    int xrow = 0, head = 0;  // key | query, its head
    bool valid = false;
    long long row_at = 0;    // queries: in lse and dsum
    float lse2 = 0.f;
    uint4 orow[kKeys ? 1 : D / 32];  // queries: this warp's quarter of the row's O
    // keys: lse and D of the step's columns, by one warp of the four that share them, a step ahead
    const bool row_warp = kKeys && (warp & 3) == 0;
    float nl = 0.f, nd = 0.f;
    // fp16: this lane's share of the largest |v|^2 of the unit's keys; keys: of |dO| and |D| of its queries
    float v_most = 0.f, g_most = 0.f, d_most = 0.f;
    auto load_row = [&](int hd, int qt) {  // head of the group and query tile
      const int q = u.a + 128 * qt + part * 32 + lane;
      const long long at = ((long long)u.b * p.H + u.h * G + hd) * p.Nq + q;
      nl = q < p.Nq ? __ldg(p.lse + at) * 1.4426950408889634f : 0.f;
      nd = q < p.Nq ? __ldcg(p.dsum + at) : 0.f;
    };
    auto open_unit = [&]() {
      xrow = kKeys ? u.x0 + r : u.x0 + (r >> p.lg_pack);
      head = kKeys ? u.h : u.h + (r & ((1 << p.lg_pack) - 1));
      valid = xrow < (kKeys ? p.Nk : p.Nq);
      if (u.n <= 0) return;
      if constexpr (!BF16) {
        const long long bh = (long long)u.b * p.Hkv + (kKeys ? u.h : u.h / G);
        const float* vm = p.vmax + bh * ((p.Nk + 127) / 128);
        // Blocks of 128, one a lane; the first 32 are not looked at here, so that nobody waits for them.
        if constexpr (kKeys) {
          v_most = __ldcg(vm + u.x0 / 128);
          const float2* qm = reinterpret_cast<const float2*>(p.qmax) + bh * ((p.Nq + 127) / 128) + u.a / 128;
          const int n = (int)((min((long long)p.Nq, u.a + 128LL * u.c) - 1) / 128) - u.a / 128 + 1;
          const float2 first = lane < n ? __ldcg(qm + lane) : make_float2(0.f, 0.f);
          g_most = first.x;
          d_most = first.y;
          for (int i = 32 + lane; i < n; i += 32) {
            const float2 w = __ldcg(qm + i);
            g_most = fmaxf(g_most, w.x);
            d_most = fmaxf(d_most, w.y);
          }
        } else {
          // the sinks' (rows of the stream below a), then those of the keys from a + c on
          const int sinks = (min(u.a, p.Nk) + 127) / 128, from = (u.a + u.c) / 128 - sinks;
          const int n = (int)((min((long long)p.Nk, 128LL * u.n + u.c) - 1) / 128) - from + 1;
          v_most = lane < n ? __ldcg(vm + (lane < sinks ? lane : from + lane)) : 0.f;
          for (int i = 32 + lane; i < n; i += 32) v_most = fmaxf(v_most, __ldcg(vm + (i < sinks ? i : from + i)));
        }
      }
      if constexpr (kKeys) {
        if (row_warp) load_row(u.s0 / u.c, u.s0 % u.c);
      } else {
        row_at = ((long long)u.b * p.H + head) * p.Nq + xrow;
        lse2 = valid ? __ldg(p.lse + row_at) : 0.f;  // in base 2 when it is used
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.o) + u.b * p.o_batch +
                                                          xrow * p.o_query + head * p.o_head + part * (D / 4));
#pragma unroll
        for (int c = 0; c < D / 32; ++c) orow[c] = valid ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    open_unit();
    for (int k = 0; u.n >= 0; ++k) {
      float dd = 0.f;  // queries: D of this lane's row
      if constexpr (!kKeys) {
        lse2 *= 1.4426950408889634f;
        if (valid && u.n == 0 && part == 0)  // a row that sees no key
          p.dsum[((long long)u.b * p.H + head) * p.Nq + xrow] = 0.f;
      }
      // fp16: dS enters its product as 2^e dS; keys: T and D times f1, dS = P' f1 (T - D)
      [[maybe_unused]] float f1 = 1.f, undo = 1.f;
      if constexpr (!BF16) {
        v_most = warp_max(v_most);
        if constexpr (kKeys) {
          const int e = ds_shift(fmaf(warp_max(g_most), sqrtf(v_most), warp_max(d_most)));
          f1 = pow2(e - kPShift);
          undo = pow2(-e);
        }
      }
      // what this lane sees: keys: queries [see_lo, see_hi); queries: keys as WindowRow
      int see_lo = 0, see_hi = 0, see_sink = 0;
      if constexpr (kKeys) {
        see_lo = (int)max(0LL, min((long long)p.Nq, xrow - diag));
        see_hi = !valid ? 0 : (xrow < p.sinks ? p.Nq : (int)max(0LL, min((long long)p.Nq, xrow - diag + p.window)));
      } else {
        const long long pos = xrow + diag;
        see_hi = valid ? (int)max(0LL, pos + 1) : 0;
        see_lo = (int)max(0LL, min((long long)p.Nk, pos - p.window + 1));
        see_sink = min(p.sinks, p.Nk);
      }
      // bits of the warp's columns of the tile whose first row is y0 that this lane sees
      auto bits = [&](int y0) -> uint32_t {
        const int at = y0 + part * 32;
        if constexpr (kKeys) return bits_below(see_hi - at, 0) & ~bits_below(see_lo - at, 0);
        else return bits_below(see_hi - at, 0) & (~bits_below(see_lo - at, 0) | bits_below(see_sink - at, 0));
      };
      int hd = 0, qt = 0;  // keys: head of the group and query tile of the step
      if (kKeys && u.n > 0) {
        hd = u.s0 / u.c;
        qt = u.s0 - hd * u.c;
      }
      for (int i = 0; i < u.n; ++i, ++g) {
        uint32_t see;
        const float* lrow = nullptr;  // keys: lse of the warp's columns; D 128 floats on
        if constexpr (kKeys) {
          see = bits(u.a + 128 * qt);
          float* buf = rowbuf + (g & 1) * 256 + part * 32;
          if (row_warp) {
            buf[lane] = BF16 ? -nl : (float)kPShift - nl;
            buf[128 + lane] = BF16 ? -nd : -nd * f1;
          }
          if (++qt == u.c) {
            qt = 0;
            ++hd;
          }
          if (row_warp && i + 1 < u.n) load_row(hd, qt);
          meet(BAR(C::kBarMeet + part), g, wctx);
          lrow = buf;
        } else {
          const int x = 128 * i;
          see = bits(x + (x >= u.a ? u.c : 0));
          if (x < u.a && x + 128 > u.a) {  // sinks, then the window
            const uint32_t sink = bits_below(u.a - x - part * 32, 0);
            see = (see & sink) | (bits(x + u.c) & ~sink);
          }
        }
        const bool all = __all_sync(0xffffffffu, see == 0xffffffffu);
        if (!kKeys && i == 0) {
          // D of the row: this warp's quarter of its channels, joined through shared memory (the
          // unit before has ended: every warp has read its D)
          mbar_wait_inline(BAR(C::kBarXFull + 1), nx & 1, wctx);
          __syncwarp();
          const uint8_t* dO = smem + C::kTile;
          float s = 0.f, n2 = 0.f;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const int chunk = part * (D / 32) + c;
            const uint4 v = *reinterpret_cast<const uint4*>(dO + (chunk >> 3) * C::kBox + r * 128 +
                                                            (((chunk & 7) ^ (r & 7)) << 4));
            const uint32_t a4[4] = {orow[c].x, orow[c].y, orow[c].z, orow[c].w}, b4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 fa = unpack2<BF16>(a4[e]), fb = unpack2<BF16>(b4[e]);
              s = fmaf(fa.x, fb.x, fmaf(fa.y, fb.y, s));
              if constexpr (!BF16) n2 = fmaf(fb.x, fb.x, fmaf(fb.y, fb.y, n2));
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(C::kBarXEmpty + 1));
          rowbuf[part * 128 + r] = s;
          [[maybe_unused]] uint8_t* norm = smem + C::kOffNorm;  // |dO|^2 of a quarter is below 2^(norm - 126)
          if constexpr (!BF16) norm[part * 128 + r] = (uint8_t)(__float_as_uint(n2) >> 23);
          meet(BAR(C::kBarMeet), nx, wctx);
          dd = (rowbuf[r] + rowbuf[128 + r]) + (rowbuf[256 + r] + rowbuf[384 + r]);
          if (valid && part == 0) p.dsum[row_at] = dd;
          if constexpr (!BF16) {
            n2 = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) n2 += pow2((int)norm[i * 128 + r] - 126);
            const float size = sqrtf(n2);
            const int e = ds_shift(fmaf(size, sqrtf(v_most), fabsf(dd)));
            undo = pow2(-e);
            lse2 -= (float)e;  // P comes out as 2^e P
            if (part == 0) {
              const float top_n = warp_max(size), top_d = warp_max(fabsf(dd));
              if (lane < 2)
                atomicMax(p.qmax + 2 * (((long long)u.b * p.Hkv + u.h / G) * ((p.Nq + 127) / 128) + u.x0 / 128) + lane,
                          __float_as_uint(lane ? top_d : top_n));
            }
          }
        }
        // ---- P
        mbar_wait_inline(BAR(C::kBarS), g & 1, wctx);
        __syncwarp();
        tc_fence_after_sync();
        float pr[32];
        {
          uint32_t s[32];
          tmem_ld32(tS, s);
          tmem_ld_wait();
          reg_order_after_wait(s);
          if constexpr (!kKeys) {  // S may be overwritten
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::kBarP));
          }
          const uint64_t cs2 = f2_make(cs, cs);
          uint64_t l2 = f2_make(-lse2, -lse2);
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            float4 l4;  // keys: of the columns, negated
            if constexpr (kKeys) l4 = *reinterpret_cast<const float4*>(lrow + c);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              if constexpr (kKeys) l2 = e ? f2_make(l4.z, l4.w) : f2_make(l4.x, l4.y);
              const float2 x = f2_split(f2_fma(f2_bits(s[c + e], s[c + e + 1]), cs2, l2));
              pr[c + e] = ex2_approx(x.x);
              pr[c + e + 1] = ex2_approx(x.y);
            }
          }
        }
        if (!all) {
#pragma unroll
          for (int c = 0; c < 32; ++c) pr[c] = seen(see, c) ? pr[c] : 0.f;
        }
        if constexpr (kKeys) {
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) w[c] = pack2<BF16>(pr[2 * c], pr[2 * c + 1]);
          tmem_st16(tS, w);  // over the first 16 of the 32 columns that this warp itself has read
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(C::kBarP));
        }
        // ---- dS
        const uint32_t tT = tS + (!kKeys && (g & 1) ? 384 : 128);
        wait_step(C::kBarT, g);
        __syncwarp();
        tc_fence_after_sync();
        {
          uint32_t t[32], w[16], rest[kKeys ? 1 : 16];
          tmem_ld32(tT, t);
          tmem_ld_wait();
          reg_order_after_wait(t);
          uint64_t d2 = f2_make(-dd, -dd);
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            float4 d4;  // keys: of the columns, negated
            if constexpr (kKeys) d4 = *reinterpret_cast<const float4*>(lrow + 128 + c);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              if constexpr (kKeys) d2 = e ? f2_make(d4.z, d4.w) : f2_make(d4.x, d4.y);
              const uint64_t td = kKeys && !BF16 ? f2_fma(f2_bits(t[c + e], t[c + e + 1]), f2_make(f1, f1), d2)
                                                 : f2_add(f2_bits(t[c + e], t[c + e + 1]), d2);
              const float2 ds = f2_split(f2_mul(f2_make(pr[c + e], pr[c + e + 1]), td));
              w[(c + e) / 2] = pack2<BF16>(ds.x, ds.y);
              if constexpr (!kKeys) {
                const float2 hi = unpack2<BF16>(w[(c + e) / 2]);
                rest[(c + e) / 2] = pack2<BF16>(ds.x - hi.x, ds.y - hi.y);
              }
            }
          }
          tmem_st16(tT, w);
          if constexpr (!kKeys) tmem_st16(tT + 16, rest);
        }
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::kBarDS + (kKeys ? 0 : g & 1)));
      }

      // ---- epilogue: this warp's quarter of the gradients' columns
      if (u.n > 0) {
        mbar_wait_inline(BAR(C::kBarAcc), nx & 1, wctx);
        ++nx;
        __syncwarp();
        tc_fence_after_sync();
      }
      const long long row = (((long long)u.b * (kKeys ? p.Nk : p.Nq) + (valid ? xrow : 0)) * (kKeys ? p.Hkv : p.H) + head) * D;
      const WindowBwdUnit done = u;
      const bool store = valid;
      u = next_unit(k + 1);
      open_unit();
#pragma unroll 1
      for (int c = part * (D / 64); c < (part + 1) * (D / 64); ++c) {  // 16 columns at a time
        uint32_t a[16], b[16];
        if (done.n > 0) {
          tmem_ld16(tmem + lane_base + 256 + c * 16, a);
          if constexpr (kKeys) tmem_ld16(tmem + lane_base + 384 + c * 16, b);
          tmem_ld_wait();
          reg_order_after_wait(a);
          if constexpr (kKeys) reg_order_after_wait(b);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) a[e] = b[e] = 0u;
        }
        // what dQ | dV and dK are to be multiplied by (but for the scale, of parts of dK)
        const float by1 = kKeys ? (BF16 ? 1.f : pow2(-kPShift)) : p.scale * undo;
        if (kKeys && done.part >= 0) {
          float4* dst = reinterpret_cast<float4*>(p.part + ((long long)done.part * 256 + r) * D + c * 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dst[e] = make_float4(__uint_as_float(a[4 * e]) * by1, __uint_as_float(a[4 * e + 1]) * by1,
                                 __uint_as_float(a[4 * e + 2]) * by1, __uint_as_float(a[4 * e + 3]) * by1);
            dst[32 * D + e] = make_float4(__uint_as_float(b[4 * e]) * undo, __uint_as_float(b[4 * e + 1]) * undo,
                                          __uint_as_float(b[4 * e + 2]) * undo, __uint_as_float(b[4 * e + 3]) * undo);
          }
        } else if (store) {
          const float by2 = p.scale * undo;
          uint4* d1 = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.g1) + row + c * 16);
          uint4* d2 = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.g2) + row + c * 16);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack2<BF16>(__uint_as_float(a[8 * e + 2 * i]) * by1, __uint_as_float(a[8 * e + 2 * i + 1]) * by1);
            d1[e] = make_uint4(w[0], w[1], w[2], w[3]);
            if constexpr (kKeys) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = pack2<BF16>(__uint_as_float(b[8 * e + 2 * i]) * by2, __uint_as_float(b[8 * e + 2 * i + 1]) * by2);
              d2[e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
      if (done.n > 0) {
        tc_fence_before_sync();  // the gradients are read before this warp's next P or dS is announced
        __syncwarp();
      }
    }
  }

  // ---- teardown: every role is done with TMEM
  tc_fence_before_sync();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// dV and dK of key tiles whose queries were split: the sum of the parts, in order.  One thread
// four channels of a key; blocks of one tile follow the units' order.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) attn_window_bwd_join_kernel(const __grid_constant__ WindowBwdParams p) {
  constexpr int kBlocks = 128 * (D / 4) / 256;
  const int heads = p.B * p.Hkv;
  int tile = blockIdx.x / kBlocks, splits, tiles, first;
  long long part;
  const int sink = p.sink_splits > 1 ? heads * p.sink_tiles : 0;  // tiles with sinks among the blocks
  if (tile < sink) {
    splits = p.sink_splits;
    tiles = p.sink_tiles;
    first = 0;
    part = (long long)tile * splits;
  } else {
    tile -= sink;
    splits = p.splits;
    tiles = p.n_xtiles - p.sink_tiles;
    first = p.sink_tiles;
    part = (long long)sink * p.sink_splits + (long long)tile * splits;
  }
  const int bh = tile / tiles, b = bh / p.Hkv, hk = bh - b * p.Hkv;
  const int e = blockIdx.x % kBlocks * 256 + threadIdx.x;
  const int r = e / (D / 4), c = e % (D / 4) * 4;
  const int key = 128 * (first + tile - bh * tiles) + r;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts have been written
  if (key >= p.Nk) return;
  float v[2][4] = {};
  for (int s = 0; s < splits; ++s)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(p.part + (((part + s) * 2 + i) * 128 + r) * D + c));
      v[i][0] += x.x;
      v[i][1] += x.y;
      v[i][2] += x.z;
      v[i][3] += x.w;
    }
  const long long row = (((long long)b * p.Nk + key) * p.Hkv + hk) * D + c;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.g1) + row) =
      make_uint2(pack2<BF16>(v[0][0], v[0][1]), pack2<BF16>(v[0][2], v[0][3]));
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.g2) + row) =
      make_uint2(pack2<BF16>(v[1][0] * p.scale, v[1][1] * p.scale), pack2<BF16>(v[1][2] * p.scale, v[1][3] * p.scale));
}

}  // namespace attn_b200
