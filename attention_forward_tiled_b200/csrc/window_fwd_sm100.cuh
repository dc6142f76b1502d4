// window_fwd_sm100.cuh -- tiled attention forward over a sliding window with sink tokens and
// grouped key/value heads (sm_100a).
//
// Query i stands at position p = i + Nk - Nq and sees key j iff j <= p and (j > p - W or
// j < S).  The kernel is the pipeline of prefill_sm100.cuh (its header describes the roles,
// barriers and TMEM layout; softmax helpers are shared) over another walk:
//   * a 128-row Q tile holds `pack` heads of one key/value group at 128 / pack consecutive
//     positions (one TMA box of pack heads x 128 / pack rows; row r is position r / pack,
//     head r % pack).  Fewer positions in a tile mean fewer key tiles that only part of it
//     sees: 256 rows of 4 heads at W = 1024 visit 1024 + 64 keys and not 1024 + 256;
//   * a unit (two Q tiles) streams the sinks (rounded up to 8 rows), then the keys from its
//     first row's lower edge to its last row's own key, as one run of 128-row tiles: a tile
//     may start at any key, and the one in which the sinks end and the window begins is put
//     together from 8-row boxes.  At W = 1024 and 4 sinks that is 9 tiles a unit, where tiles
//     cut at multiples of 128 keys came to 10.5 on average (411 us, against 360 us).  Tile 1
//     leaves out stream tiles that lie below its window where there are no sinks (at most one:
//     its positions start 128 / pack later);
//   * a unit of one Q tile (where pairs would leave SMs without work) gives both tile slots the
//     same rows: slot 0 takes the even stream tiles, slot 1 the odd ones, each with its own
//     maximum, sum and O, and slot 0's warps join the two from TMEM at the end.  So one tile
//     overlaps softmax and products as two do (500 queries of 32 heads over 2000 keys each:
//     39 us with an idle slot, 35 us so);
//   * a tile that the window, the sinks' end or the diagonal cuts is masked by a 128-bit
//     row mask; every other tile takes the unmasked path.
// What bounds it is what bounds the causal forward: exponentials and the S -> P -> P V chain
// of the tensor cores.  4096 queries of 4 x 32 heads over 8, 128 channels, W = 1024: 335 us, in
// which the tensor cores work 39 % and the exponential unit 39 %.
#pragma once

#include "prefill_sm100.cuh"

namespace attn_b200 {

struct WindowFwdParams {
  CUtensorMap tm_q;  // [B, Nq, H, D] as 4-D (D, H, Nq, B), box (64, pack, 128 / pack, 1), 128B swizzle
  CUtensorMap tm_k;  // [B, Nk, Hkv, D], box (64, 1, 128, 1)
  CUtensorMap tm_v;  // same
  CUtensorMap tm_k8; // as tm_k, box (64, 1, 8, 1)
  CUtensorMap tm_v8; // same
  CUtensorMap tm_o;  // as tm_q (store)
  void* out;         // raw output pointer (rows that see no key are written directly)
  float* lse;        // [B, H, Nq] or nullptr
  int* status;
  int B, H, Nq, Nk;
  int group;         // query heads of a key/value head
  int lg_pack;       // log2 of the heads in a Q tile (pack divides group)
  int window, sinks;
  int n_pairs;       // Q tile pairs along the queries: ceil(Nq / (256 / pack))
  int n_split;       // the last n_split pair units run as two units of one tile each
  float scale_log2;  // scale * log2(e)
  unsigned long long timeout_ns;
  int inject;        // test hook: 1 = the first Q tile never counts as landed
};

constexpr int kWindowUnitInts = 10;  // ints per published work unit (WindowUnit)

template <int D>
struct WindowFwdCfg : PrefillCfg<D> {
  using Base = PrefillCfg<D>;
  static constexpr int kMiscBytes = 16 + 2 * kWindowUnitInts * 4;
  static constexpr int kOffClc = ((Base::kOffMisc + kMiscBytes + 15) / 16) * 16;
  static_assert(kOffClc + 16 <= Base::kBarBytes, "barrier area too small");
  static constexpr int kOffMl = Base::kOffBar + Base::kBarBytes;  // float2 [128]: slot 1's maxima and sums
  static constexpr int kOffJoin = kOffMl + 1024;  // barriers: slot 1's rows are there, (d = 64) slot 0 has read them
  static constexpr int kSmemBytes = Base::kSmemBytes + 1024 + 16;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

// kShared: units whose two slots share a Q tile occur.
template <bool kShared>
struct WindowUnit {
  int b, h;         // batch, first head of the Q tiles
  int pos0[2];      // first query of each tile
  int end[2];       // one past each tile's last stream tile (0: no row of the tile sees a key)
  int nmax;         // stream tiles (-1: no more units)
  int sink8;        // stream rows 0 .. sink8 - 1 (a multiple of 8) are keys 0 .. sink8 - 1,
  int shift;        // stream row x from there on is key x + shift
  int skip1;        // leading stream tiles that Q tile 1 leaves out; -1: one Q tile in both slots
  __device__ __forceinline__ bool shared() const { return kShared && skip1 < 0; }
  __device__ __forceinline__ bool active(int t, int j) const {
    return j < end[t] && (shared() ? (j & 1) == t : (t == 0 || j >= skip1));
  }
  // stream tile j is the first that slot t takes part in
  __device__ __forceinline__ bool starts(int t, int j) const { return j == (t == 0 ? 0 : shared() ? 1 : skip1); }
  // stream tiles from one of a slot's to its next
  __device__ __forceinline__ int ahead() const { return shared() ? 2 : 1; }
  // key of stream tile j's first row, and of its rows from the sinks' end on
  __device__ __forceinline__ int key0(int j) const { return 128 * j + (128 * j >= sink8 ? shift : 0); }
  __device__ __forceinline__ bool mixed(int j) const { return 128 * j < sink8 && 128 * j + 128 > sink8; }
};

// The warps that `bar` counts meet there for the n-th time.  Unlike a named barrier the wait ends
// when the kernel is given up, which its warps may learn at different units.
__device__ __forceinline__ void meet(uint32_t bar, int n, const WaitCtx& wctx) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
  mbar_wait_inline(bar, n & 1, wctx);
  __syncwarp();
}

// Unit index -> batch, heads, queries and key tiles.  Units run along the queries of a head
// block first, so the K/V in use stay in L2.
template <bool kShared>
__device__ __forceinline__ WindowUnit<kShared> window_unit(const WindowFwdParams& p, int unit) {
  const int pack = 1 << p.lg_pack, rows = 128 >> p.lg_pack;  // heads, positions of a Q tile
  const int blocks = p.H >> p.lg_pack;                       // head blocks of a batch
  const int n_pairs = p.B * blocks * p.n_pairs - p.n_split;
  int pair = unit, single = -1;  // single: which tile of a split pair this unit runs
  if (kShared && unit >= n_pairs) {
    pair = n_pairs + ((unit - n_pairs) >> 1);
    single = (unit - n_pairs) & 1;
  }
  const int bh = pair / p.n_pairs, qp = pair - bh * p.n_pairs;
  WindowUnit<kShared> u;
  u.b = bh / blocks;
  u.h = (bh - u.b * blocks) * pack;
  u.pos0[0] = qp * 2 * rows + (single == 1 ? rows : 0);
  u.pos0[1] = u.pos0[0] + (single >= 0 ? 0 : rows);
  long long lo[2], hi[2];  // first key and last key of each Q tile's window (hi < 0: none)
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const long long pos = (long long)u.pos0[t] + p.Nk - p.Nq;  // position of the first query
    const int count = min(rows, p.Nq - u.pos0[t]);
    lo[t] = max(0LL, pos - p.window + 1);
    hi[t] = count > 0 ? pos + count - 1 : -1;
  }
  int low = (int)(hi[0] >= 0 ? lo[0] : lo[1]);
  u.sink8 = (int)min(((long long)p.sinks + 7) / 8 * 8, 1LL << 30);
  if (u.sink8 >= low) u.sink8 = low = 0;  // the sinks reach the window: one run of keys from 0
  u.shift = low - u.sink8;
  u.skip1 = (hi[0] >= 0 && hi[1] >= 0 && u.sink8 == 0 && p.sinks <= low) ? (int)((lo[1] - low) / 128) : 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) u.end[t] = hi[t] >= 0 ? ((int)hi[t] - u.shift) / 128 + 1 : 0;
  if (single >= 0) {
    u.skip1 = -1;
    const int n = u.end[0];  // stream tiles: the even ones are slot 0's
    u.end[0] = n - (n > 0 && n % 2 == 0 ? 1 : 0);
    u.end[1] = n > 1 ? n - n % 2 : 0;
  }
  u.nmax = max(u.end[0], u.end[1]);
  return u;
}

// Bits of word w (of 4) below n.
__device__ __forceinline__ uint32_t bits_below(int n, int w) {
  n -= 32 * w;
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

// What one row of a Q tile sees.
struct WindowRow {
  int lim;             // keys below lim
  int lo, sinks;       // and at or past lo, or below sinks
  int lim_min, lo_max; // the same edges of the row of the tile that cuts most
  __device__ __forceinline__ bool cuts(int key0) const {
    return key0 + 128 > lim_min || (key0 < lo_max && key0 + 128 > sinks);
  }
  __device__ __forceinline__ uint32_t word(int key0, int w) const {
    return bits_below(lim - key0, w) & (~bits_below(lo - key0, w) | bits_below(sinks - key0, w));
  }
  // Whether some row of the Q tile does not see all of stream tile j, and this row's bits of it.
  template <bool kShared>
  __device__ __forceinline__ bool masked(const WindowUnit<kShared>& u, int j, uint32_t (&see)[4]) const {
    const int key0 = u.key0(j);
    const bool mixed = u.mixed(j);
    if (!mixed && !cuts(key0)) return false;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      see[w] = word(key0, w);
      if (mixed) {
        const uint32_t head = bits_below(u.sink8 - 128 * j, w);
        see[w] = (see[w] & head) | (word(key0 + u.shift, w) & ~head);
      }
    }
    return true;
  }
};

// Positions lie in (-2^31, 2^31); rows past Nq count as the last key's position.
__device__ __forceinline__ WindowRow window_row(const WindowFwdParams& p, int pos0, int query) {
  const long long diag = (long long)p.Nk - p.Nq;
  const long long pos = min((long long)query + diag, (long long)p.Nk - 1);
  const long long low = (long long)pos0 + diag;
  const long long high = min(low + (128 >> p.lg_pack) - 1, (long long)p.Nk - 1);
  WindowRow r;
  r.lim = (int)max(0LL, pos + 1);
  r.lo = (int)max(0LL, pos - p.window + 1);
  r.sinks = min(p.sinks, p.Nk);
  r.lim_min = (int)max(0LL, low + 1);
  r.lo_max = (int)max(0LL, high - p.window + 1);
  return r;
}

__device__ __forceinline__ bool seen(uint32_t word, int c) { return (word >> (c & 31)) & 1u; }

// half_max and row_max of prefill_sm100.cuh over the keys whose bit is set.
template <bool kNeg, int kHalf>
__device__ __forceinline__ float seen_half_max(const uint32_t (&h)[2][32], const uint32_t (&see)[4]) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < 64; c += 2) {
    const float s0 = __uint_as_float(h[c >> 5][c & 31]), s1 = __uint_as_float(h[c >> 5][(c & 31) + 1]);
    const uint32_t w = see[2 * kHalf + (c >> 5)];
    m[(c >> 1) & 3] = fmax3(m[(c >> 1) & 3], seen(w, c) ? (kNeg ? -s0 : s0) : -INFINITY,
                            seen(w, c + 1) ? (kNeg ? -s1 : s1) : -INFINITY);
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// p = 2^(cs s - m_use) for one 64-column half (0 where a bit of `see` is not set, when kMask),
// packed into 32 fp16 pairs; returns their sum, and in xmax the largest exponent.  The sum is of
// the fp32 values, before P is rounded for the product, and every exponential is the hardware's
// (2^-22): the log-sum-exp keeps fp32's precision.
template <bool kMask, int kHalf>
__device__ __forceinline__ float window_half_exp(const uint32_t (&h)[2][32], float cs, float m_use,
                                                 const uint32_t (&see)[4], uint32_t (&pk)[32], float& xmax) {
  uint64_t acc[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
  float mx[2] = {xmax, -INFINITY};
  const uint64_t cs2 = f2_make(cs, cs), negm2 = f2_make(-m_use, -m_use);
#pragma unroll
  for (int c = 0; c < 64; c += 2) {
    float2 x = f2_split(f2_fma(
        f2_make(__uint_as_float(h[c >> 5][c & 31]), __uint_as_float(h[c >> 5][(c & 31) + 1])), cs2, negm2));
    if (kMask) {
      const uint32_t w = see[2 * kHalf + (c >> 5)];
      x.x = seen(w, c) ? x.x : -INFINITY;
      x.y = seen(w, c + 1) ? x.y : -INFINITY;
    }
    mx[(c >> 1) & 1] = fmax3(mx[(c >> 1) & 1], x.x, x.y);
    const float2 pp = make_float2(ex2_approx(x.x), ex2_approx(x.y));
    acc[(c >> 1) & 1] = f2_add(acc[(c >> 1) & 1], f2_make(pp.x, pp.y));
    pk[c >> 1] = pack2<false>(pp.x, pp.y);
  }
  xmax = fmaxf(mx[0], mx[1]);
  const float2 sum = f2_split(f2_add(acc[0], acc[1]));
  return sum.x + sum.y;
}

template <bool kNeg>
__device__ __forceinline__ float seen_row_max(const uint32_t (&sr)[4][32], const uint32_t (&see)[4]) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < 128; c += 2) {
    const float s0 = __uint_as_float(sr[c >> 5][c & 31]), s1 = __uint_as_float(sr[c >> 5][(c & 31) + 1]);
    m[(c >> 1) & 3] = fmax3(m[(c >> 1) & 3], seen(see[c >> 5], c) ? (kNeg ? -s0 : s0) : -INFINITY,
                            seen(see[c >> 5], c + 1) ? (kNeg ? -s1 : s1) : -INFINITY);
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// The same for the whole row (d = 64), stored into 64 TMEM columns from tP on.
template <bool kMask>
__device__ __forceinline__ float window_row_exp_to_tmem(const uint32_t (&sr)[4][32], float cs, float m_use,
                                                        const uint32_t (&see)[4], uint32_t tP) {
  uint64_t acc[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
  const uint64_t cs2 = f2_make(cs, cs), negm2 = f2_make(-m_use, -m_use);
#pragma unroll
  for (int q32 = 0; q32 < 4; ++q32) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int c = q32 * 32 + 2 * i;
      const float2 x = f2_split(
          f2_fma(f2_make(__uint_as_float(sr[q32][2 * i]), __uint_as_float(sr[q32][2 * i + 1])), cs2, negm2));
      float2 pp = make_float2(ex2_approx(x.x), ex2_approx(x.y));
      if (kMask) {
        pp.x = seen(see[q32], c) ? pp.x : 0.f;
        pp.y = seen(see[q32], c + 1) ? pp.y : 0.f;
      }
      acc[i & 1] = f2_add(acc[i & 1], f2_make(pp.x, pp.y));
      w[i] = pack2<false>(pp.x, pp.y);
    }
    tmem_st16(tP + q32 * 16, w);
  }
  const float2 sum = f2_split(f2_add(acc[0], acc[1]));
  return sum.x + sum.y;
}

// Slot 0's warps of a unit that both slots share, the n-th: m and l become those of both slots'
// keys, and returned is what O_0 is to be multiplied by, in f1 what O_1 is.  Other units: 1 / l.
template <bool kShared>
__device__ __forceinline__ float join_slots(const WindowUnit<kShared>& u, const float2* slot1, int r, float& m, float& l,
                                            float& f1, uint32_t join, int n, const WaitCtx& wctx) {
  float a0 = 1.f;
  if (u.shared()) {
    mbar_wait_inline(join, n & 1, wctx);
    __syncwarp();
    tc_fence_after_sync();
    const float2 x = slot1[r];
    const float top = fmaxf(m, x.x), use = top == -INFINITY ? 0.f : top;
    a0 = ex2_approx(m - use);
    f1 = ex2_approx(x.x - use);
    l = fmaf(a0, l, f1 * x.y);
    m = top;
  }
  const float inv_l = l > 0.f ? 1.0f / l : 0.f;
  f1 *= inv_l;
  return a0 * inv_l;
}

// The row f0 O_0 + f1 O_1 (TMEM columns from tO0 and tO1 on) to the staging buffer, 32 columns at
// a time; O_1 may be overwritten then.
template <int D, bool BF16, bool kShared>
__device__ __forceinline__ void stage_joined(const WindowUnit<kShared>& u, uint32_t tO0, uint32_t tO1, float f0, float f1,
                                             uint8_t* stage, int r, uint32_t join) {
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t o[32], x[32];
    tmem_ld32(tO0 + c * 32, o);
    if (u.end[1] > 0) tmem_ld32(tO1 + c * 32, x);
    tmem_ld_wait();
    reg_order_after_wait(o);
    if (u.end[1] > 0) reg_order_after_wait(x);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const float v = __uint_as_float(o[e]) * f0;
      o[e] = __float_as_uint(u.end[1] > 0 ? fmaf(__uint_as_float(x[e]), f1, v) : v);
    }
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = pack2<BF16>(__uint_as_float(o[q4 * 8 + 2 * i]), __uint_as_float(o[q4 * 8 + 2 * i + 1]));
      const int chunk = c * 4 + q4, bx = chunk >> 3, cc = chunk & 7;
      *reinterpret_cast<uint4*>(stage + bx * PrefillCfg<D>::kBoxBytes + r * 128 + ((cc ^ (r & 7)) << 4)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  tc_fence_before_sync();
  __syncwarp();
  // d = 128: the turn with the staging buffer says so
  if (D == 64 && (threadIdx.x & 31) == 0) mbar_arrive(join + 8);
}

template <int D, bool BF16, bool kShared>
__global__ void __launch_bounds__(WindowFwdCfg<D>::kThreads, 1)
    attn_window_fwd_kernel(const __grid_constant__ WindowFwdParams p) {
  using C = WindowFwdCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t sbase = (raw_addr + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw_addr);

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* unit_slot = reinterpret_cast<volatile int*>(tmem_slot + 4);  // [2][kWindowUnitInts]
  const uint32_t clc_resp = sbase + C::kOffBar + C::kOffClc;
  float2* slot1 = reinterpret_cast<float2*>(smem + C::kOffMl);
  auto BAR = [&](int i) -> uint32_t { return smem_u32(&bars[i]); };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const WaitCtx wctx{abort_flag, p.status, p.timeout_ns};
  const uint32_t join = sbase + C::kOffJoin;

  // ---- one-time setup
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(C::kBarQFull + i), p.inject == 1 && i == 0 ? 2 : 1);
      mbar_init(BAR(C::kBarQEmpty + i), 1);
      mbar_init(BAR(C::kBarSFull + i), 1);
      mbar_init(BAR(C::kBarSFree + i), 4);  // one arrive per softmax warp
      mbar_init(BAR(C::kBarPFull + i), 4);  // one arrive per softmax warp
      mbar_init(BAR(C::kBarPVDone + i), 1);
      mbar_init(BAR(C::kBarUnitFull + i), 1);
      mbar_init(BAR(C::kBarUnitEmpty + i), C::kUnitReaders);
      mbar_init(BAR(C::kBarOStage + i), 4);  // one arrive per softmax warp
      mbar_init(BAR(C::kBarOReady + i), 4);  // one arrive per softmax warp
      mbar_init(BAR(C::kBarOFree + i), 1);
      mbar_init(BAR(C::kBarPHalf + i), 4);  // one arrive per softmax warp
    }
    mbar_init(join, 4);  // one arrive per softmax warp of slot 1
    mbar_init(join + 8, 4);  // and of slot 0
    mbar_init(BAR(C::kBarMmaDone), 1);
    mbar_init(BAR(C::kBarClc), 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(BAR(C::kBarKVFull + s), 1);
      // bf16: the two converter warps also observe and release every ring item, so no
      // waiter on these barriers can ever be two phases behind or ahead
      mbar_init(BAR(C::kBarKVEmpty + s), BF16 ? 3 : 1);
      mbar_init(BAR(C::kBarVConv + s), 2);  // one arrive per converter warp, every ring item
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  // Every role walks the same unit sequence, decoded and published by the producer.
  // Returns the k-th unit (nmax < 0: no more) after this warp has read it and released
  // its slot.
  using Unit = WindowUnit<kShared>;
  auto next_unit = [&](int k) -> Unit {
    mbar_wait_inline(BAR(C::kBarUnitFull + (k & 1)), (k >> 1) & 1, wctx);
    __syncwarp();
    const volatile int* us = unit_slot + (k & 1) * kWindowUnitInts;
    Unit u;
    u.b = us[0];
    u.h = us[1];
    u.pos0[0] = us[2];
    u.pos0[1] = us[3];
    u.end[0] = us[4];
    u.end[1] = us[5];
    u.nmax = us[6];
    u.sink8 = us[7];
    u.shift = us[8];
    u.skip1 = us[9];
    if (warp_flag(abort_flag)) u.nmax = -1;  // a slot read after a wait that gave up may be stale
    __syncwarp();
    if (lane == 0) mbar_arrive(BAR(C::kBarUnitEmpty + (k & 1)));
    return u;
  };

  static_assert(C::kProducerWarp == 8 && C::kMmaWarp == 9 && C::kConvWarp0 == 10 && C::kThreads == 384,
                "warpgroup 2 = producer, MMA issuer, two converter warps");
  // Roles.  setmaxnreg must dominate the code it governs, so each warpgroup's re-balance
  // (d = 64) opens its branch and the return to the launch's count closes it.
  if (warp >= C::kProducerWarp) {
    // warpgroup 2: producer, MMA issuer, converters
    if constexpr (C::kDecoupled) warpgroup_reg_dealloc<C::kRegsAux>();
    if (warp == C::kProducerWarp) {
      // ======================= producer: unit claims + TMA loads ======================
      if (lane == 0) {
        tma_prefetch_map(&p.tm_q);
        tma_prefetch_map(&p.tm_k);
        tma_prefetch_map(&p.tm_v);
        tma_prefetch_map(&p.tm_o);
      }
      __syncwarp();
      int unit = blockIdx.x;  // the first unit is this CTA's own
      int nq[2] = {0, 0};     // Q loads issued per tile
      bool q_pending[2] = {false, false};
      int g = 0;              // ring items issued
      int nclaim = 0;
      for (int k = 0;; ++k) {
        Unit u;
        if (unit >= 0) {
          u = window_unit<kShared>(p, unit);
        } else {
          u.b = u.h = u.pos0[0] = u.pos0[1] = u.end[0] = u.end[1] = u.sink8 = u.shift = u.skip1 = 0;
          u.nmax = -1;
        }
        if (k >= 2) mbar_wait_inline(BAR(C::kBarUnitEmpty + (k & 1)), ((k >> 1) - 1) & 1, wctx);
        __syncwarp();
        if (lane == 0) {
          volatile int* us = unit_slot + (k & 1) * kWindowUnitInts;
          us[0] = u.b;
          us[1] = u.h;
          us[2] = u.pos0[0];
          us[3] = u.pos0[1];
          us[4] = u.end[0];
          us[5] = u.end[1];
          us[6] = u.nmax;
          us[7] = u.sink8;
          us[8] = u.shift;
          us[9] = u.skip1;
          mbar_arrive(BAR(C::kBarUnitFull + (k & 1)));
        }
        __syncwarp();
        if (unit < 0) break;
        // The next unit is claimed late in this one (kClaimLead ring items before its last
        // load), so units go to the CTAs that are about to run out of work: claiming a
        // whole unit ahead leaves a tail of up to one long causal unit between SMs.
        bool claimed = false;
        const int claim_at = max(0, 2 * u.nmax - C::kClaimLead);
        auto claim_next = [&]() {
          if (!claimed && !warp_flag(abort_flag)) {
            mbar_arrive_expect_tx_w(BAR(C::kBarClc), 16);
            clc_try_cancel_w(clc_resp, BAR(C::kBarClc));
            claimed = true;
          }
        };
        for (int t = 0; t < 2; ++t) {
          if (u.end[t] == 0) continue;
          if (nq[t] > 0) mbar_wait_inline(BAR(C::kBarQEmpty + t), (nq[t] - 1) & 1, wctx);
          __syncwarp();
          if (!warp_flag(abort_flag)) {
            mbar_arrive_expect_tx_w(BAR(C::kBarQFull + t), C::kTileBytes);
            for (int bx = 0; bx < C::kBoxes; ++bx)
              tma_load_4d_w(sbase + C::kOffQ + t * C::kTileBytes + bx * C::kBoxBytes, &p.tm_q,
                            BAR(C::kBarQFull + t), bx * 64, u.h, u.pos0[t], u.b);
            q_pending[t] = true;
          }
          ++nq[t];
        }
        const int kv_head = u.h / p.group;
        for (int i = 0; i < 2 * u.nmax; ++i, ++g) {
          if (i == claim_at) claim_next();
          const int stage = g % C::kStages;
          const int round = g / C::kStages;
          if (round > 0) mbar_wait_inline(BAR(C::kBarKVEmpty + stage), (round - 1) & 1, wctx);
          __syncwarp();
          if (warp_flag(abort_flag)) continue;
          mbar_arrive_expect_tx_w(BAR(C::kBarKVFull + stage), C::kTileBytes);
          const uint32_t dst = sbase + C::kOffKV + stage * C::kTileBytes;
          const int key0 = u.key0(i >> 1);
          if (!u.mixed(i >> 1)) {
            const CUtensorMap* map = (i & 1) ? &p.tm_v : &p.tm_k;
            for (int bx = 0; bx < C::kBoxes; ++bx)
              tma_load_4d_w(dst + bx * C::kBoxBytes, map, BAR(C::kBarKVFull + stage), bx * 64, kv_head, key0, u.b);
          } else if (lane < 16) {
            // lane l copies rows 8 l .. 8 l + 7 of the tile (one 1 KB swizzle atom a box)
            const CUtensorMap* map = (i & 1) ? &p.tm_v8 : &p.tm_k8;
            const int key = key0 + 8 * lane + (key0 + 8 * lane >= u.sink8 ? u.shift : 0);
            for (int bx = 0; bx < C::kBoxes; ++bx)
              tma_load_4d(dst + bx * C::kBoxBytes + lane * 1024, map, BAR(C::kBarKVFull + stage), bx * 64, kv_head, key,
                          u.b);
          }
          __syncwarp();
        }
        claim_next();  // units without K/V tiles
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
        // Let every copy this warp started land before the CTA can exit.
        for (int t = 0; t < 2; ++t)
          if (q_pending[t]) mbar_wait_drain_inline(BAR(C::kBarQFull + t), (nq[t] - 1) & 1, p.timeout_ns);
        const int first = g > C::kStages ? g - C::kStages : 0;
        for (int i = first; i < g; ++i)
          mbar_wait_drain_inline(BAR(C::kBarKVFull + i % C::kStages), (i / C::kStages) & 1, p.timeout_ns);
        __syncwarp();
      }
    } else if (warp == C::kMmaWarp) {
      if constexpr (C::kDecoupled) {
      // ======================= tcgen05 MMA issuer (one elected lane issues) ===========
      constexpr uint32_t idesc_s = make_idesc_f16(128, 128, BF16, false);  // Q K^T, both K-major
      // P V always runs in fp16 (bf16 V tiles are converted in shared memory first); V is MN-major
      constexpr uint32_t idesc_o = make_idesc_f16(128, D, false, true);
      const uint32_t colS[2] = {0u, 128u};
      const uint32_t colO[2] = {256u, 256u + D};
      const uint32_t sQ[2] = {sbase + C::kOffQ, sbase + C::kOffQ + C::kTileBytes};
      // S_t = Q_t K_j^T: the D / 16 = 4 k-steps of 16 elements (32 bytes apart inside the
      // 128-byte swizzle rows of one box), issued in one batch.
      static_assert(D == 64, "the decoupled pipeline runs at head_dim 64");
      auto issue_s = [&](int t, uint32_t sK) {
        mma_f16_ss_k64_w(tmem + colS[t], make_sdesc_sw128(sQ[t], 16, 1024), make_sdesc_sw128(sK, 16, 1024),
                         idesc_s, 0u);
      };
      // O_t += P_t V_j over 8 k-steps of 16 keys (P_t in its own TMEM columns), issued in two
      // batches of four.
      auto issue_pv = [&](int t, uint32_t sV, bool accumulate_first) {
        mma_f16_ts_k64_w<2048>(tmem + colO[t], tmem + C::kColP + 64 * t,
                               make_sdesc_sw128(sV, C::kBoxBytes, 1024), idesc_o, accumulate_first ? 1u : 0u);
        mma_f16_ts_k64_w<2048>(tmem + colO[t], tmem + C::kColP + 64 * t + 32,
                               make_sdesc_sw128(sV + 4 * 2048, C::kBoxBytes, 1024), idesc_o, 1u);
      };
      auto stage_addr = [&](int item) -> uint32_t {
        return sbase + C::kOffKV + (item % C::kStages) * C::kTileBytes;
      };
      int nq[2] = {0, 0};   // units seen per tile (q_full / q_empty phases)
      int nsf[2] = {0, 0};  // S tiles released by the softmax (s_free phases)
      int npf[2] = {0, 0};  // P tiles written by the softmax (p_full phases)
      int g = 0;            // ring items consumed
      for (int k = 0;; ++k) {
        const Unit u = next_unit(k);
        if (u.nmax < 0) break;
        if (u.nmax == 0) continue;
        for (int t = 0; t < 2; ++t)
          if (u.end[t] > 0) mbar_wait_inline(BAR(C::kBarQFull + t), nq[t] & 1, wctx);
        // prologue: each slot's first S
        const int ahead = u.ahead();
        for (int j = 0; j < min(ahead, u.nmax); ++j) {
          const int ik = g + 2 * j;  // ring item of K_j
          mbar_wait_inline(BAR(C::kBarKVFull + ik % C::kStages), (ik / C::kStages) & 1, wctx);
          __syncwarp();
          tc_fence_after_sync();
          if (warp_flag(abort_flag)) continue;
          for (int t = 0; t < 2; ++t)
            if (u.active(t, j)) {
              issue_s(t, stage_addr(ik));
              tc_commit_w(BAR(C::kBarSFull + t));
              if (u.end[t] == j + 1) tc_commit_w(BAR(C::kBarQEmpty + t));
            }
          tc_commit_w(BAR(C::kBarKVEmpty + ik % C::kStages));
        }
        for (int j = 0; j < u.nmax; ++j) {
          // next score tiles: S_t(j+1) as soon as the softmax has read S_t(j) out of TMEM
          const int ik = g + 2 * (j + ahead);  // ring item of the slots' next K
          bool k_ready = false;
          for (int t = 0; t < 2; ++t) {
            if (u.active(t, j)) {
              mbar_wait_inline(BAR(C::kBarSFree + t), nsf[t] & 1, wctx);
              ++nsf[t];
              __syncwarp();
            }
            if (u.active(t, j + ahead)) {
              if (!k_ready) {
                mbar_wait_inline(BAR(C::kBarKVFull + ik % C::kStages), (ik / C::kStages) & 1, wctx);
                __syncwarp();
                k_ready = true;
              }
              tc_fence_after_sync();
              if (warp_flag(abort_flag)) continue;
              issue_s(t, stage_addr(ik));
              tc_commit_w(BAR(C::kBarSFull + t));
              if (j + ahead + 1 == u.end[t]) tc_commit_w(BAR(C::kBarQEmpty + t));
            }
          }
          if (k_ready && !warp_flag(abort_flag)) tc_commit_w(BAR(C::kBarKVEmpty + ik % C::kStages));
          // O_t += P_t(j) V_j once the softmax has written P_t(j)
          const int iv = g + 2 * j + 1;  // ring item of V_j
          mbar_wait_inline(BAR((BF16 ? C::kBarVConv : C::kBarKVFull) + iv % C::kStages), (iv / C::kStages) & 1,
                    wctx);
          __syncwarp();
          for (int t = 0; t < 2; ++t) {
            if (!u.active(t, j)) continue;
            mbar_wait_inline(BAR(C::kBarPFull + t), npf[t] & 1, wctx);
            ++npf[t];
            __syncwarp();
            tc_fence_after_sync();
            if (warp_flag(abort_flag)) continue;
            issue_pv(t, stage_addr(iv), !u.starts(t, j));
            tc_commit_w(BAR(C::kBarPVDone + t));
          }
          if (!warp_flag(abort_flag)) tc_commit_w(BAR(C::kBarKVEmpty + iv % C::kStages));
        }
        g += 2 * u.nmax;
        for (int t = 0; t < 2; ++t)
          if (u.end[t] > 0) ++nq[t];
      }
      // every MMA (and every commit arrive) has landed before TMEM is released
      tc_commit_w(BAR(C::kBarMmaDone));
      mbar_wait_drain_inline(BAR(C::kBarMmaDone), 0, p.timeout_ns);
      __syncwarp();
      } else {
      // ======================= tcgen05 MMA issuer (one elected lane issues) ===========
      constexpr uint32_t idesc_s = make_idesc_f16(128, 128, BF16, false);  // Q K^T, both K-major
      // P V always runs in fp16 (bf16 V tiles are converted in shared memory first); V is MN-major
      constexpr uint32_t idesc_o = make_idesc_f16(128, D, false, true);
      const uint32_t colS[2] = {0u, 128u};
      const uint32_t colO[2] = {256u, 256u + D};
      const uint32_t sQ[2] = {sbase + C::kOffQ, sbase + C::kOffQ + C::kTileBytes};
      // S_t = Q_t K_j^T over D/16 k-steps of 16 elements (32 bytes inside a 128-byte swizzle row).
      // S_t = Q_t K_j^T: 8 k-steps of 16 elements, issued in one batch.
      auto issue_s = [&](int t, uint32_t sK) {
        mma_f16_ss_k128_w<C::kBoxBytes>(tmem + colS[t], make_sdesc_sw128(sQ[t], 16, 1024),
                                        make_sdesc_sw128(sK, 16, 1024), idesc_s, 0u);
      };
      // k-steps kk0 .. kk0+3 of O_t += P_t V_j (keys 16*kk0 .. 16*kk0+63; P_t is in TMEM
      // columns [64,128) of S_t), issued in one batch; the first k-step of the unit starts
      // the accumulator.
      auto issue_pv4 = [&](int t, uint32_t sV, int kk0, bool accumulate_first) {
        mma_f16_ts_k64_w<2048>(tmem + colO[t], tmem + colS[t] + 64 + kk0 * 8,
                               make_sdesc_sw128(sV + kk0 * 2048, C::kBoxBytes, 1024), idesc_o,
                               accumulate_first ? 1u : 0u);
      };
      auto stage_addr = [&](int item) -> uint32_t {
        return sbase + C::kOffKV + (item % C::kStages) * C::kTileBytes;
      };
      int nq[2] = {0, 0};  // units seen per tile (q_full / q_empty phases)
      int np[2] = {0, 0};  // P tiles consumed per tile (p_ready phases)
      int g = 0;           // ring items consumed
      for (int k = 0;; ++k) {
        const Unit u = next_unit(k);
        if (u.nmax < 0) break;
        if (u.nmax == 0) continue;
        for (int t = 0; t < 2; ++t)
          if (u.end[t] > 0) mbar_wait_inline(BAR(C::kBarQFull + t), nq[t] & 1, wctx);
        // prologue: each slot's first S
        const int ahead = u.ahead();
        for (int j = 0; j < min(ahead, u.nmax); ++j) {
          const int ik = g + 2 * j;  // ring item of K_j
          mbar_wait_inline(BAR(C::kBarKVFull + ik % C::kStages), (ik / C::kStages) & 1, wctx);
          __syncwarp();
          tc_fence_after_sync();
          if (warp_flag(abort_flag)) continue;
          for (int t = 0; t < 2; ++t)
            if (u.active(t, j)) {
              issue_s(t, stage_addr(ik));
              tc_commit_w(BAR(C::kBarSFull + t));
              if (u.end[t] == j + 1) tc_commit_w(BAR(C::kBarQEmpty + t));
            }
          tc_commit_w(BAR(C::kBarKVEmpty + ik % C::kStages));
        }
        for (int j = 0; j < u.nmax; ++j) {
          const int iv = g + 2 * j + 1;  // ring item of V_j
          mbar_wait_inline(BAR((BF16 ? C::kBarVConv : C::kBarKVFull) + iv % C::kStages), (iv / C::kStages) & 1,
                    wctx);
          __syncwarp();
          const int ik = g + 2 * (j + ahead);  // ring item of the slots' next K
          bool k_ready = false;
          for (int t = 0; t < 2; ++t) {
            if (u.active(t, j)) {
              // keys 64..127 as soon as that half of P_t(j) is written, then keys 0..63
              mbar_wait_inline(BAR(C::kBarPHalf + t), np[t] & 1, wctx);
              __syncwarp();
              tc_fence_after_sync();
              if (!warp_flag(abort_flag)) issue_pv4(t, stage_addr(iv), 4, !u.starts(t, j));
              mbar_wait_inline(BAR(C::kBarPFull + t), np[t] & 1, wctx);
              ++np[t];
              __syncwarp();
              tc_fence_after_sync();
              if (warp_flag(abort_flag)) continue;
              issue_pv4(t, stage_addr(iv), 0, true);
              if (j + 1 == u.end[t]) tc_commit_w(BAR(C::kBarPVDone + t));
            }
            if (u.active(t, j + ahead)) {
              if (!k_ready) {
                mbar_wait_inline(BAR(C::kBarKVFull + ik % C::kStages), (ik / C::kStages) & 1, wctx);
                __syncwarp();
                k_ready = true;
              }
              if (warp_flag(abort_flag)) continue;
              issue_s(t, stage_addr(ik));
              tc_commit_w(BAR(C::kBarSFull + t));
              if (j + ahead + 1 == u.end[t]) tc_commit_w(BAR(C::kBarQEmpty + t));
            }
          }
          if (!warp_flag(abort_flag)) {
            tc_commit_w(BAR(C::kBarKVEmpty + iv % C::kStages));
            if (k_ready) tc_commit_w(BAR(C::kBarKVEmpty + ik % C::kStages));
          }
        }
        g += 2 * u.nmax;
        for (int t = 0; t < 2; ++t)
          if (u.end[t] > 0) ++nq[t];
      }
      // every MMA (and every commit arrive) has landed before TMEM is released
      tc_commit_w(BAR(C::kBarMmaDone));
      mbar_wait_drain_inline(BAR(C::kBarMmaDone), 0, p.timeout_ns);
      __syncwarp();
      }
    } else if (warp >= C::kConvWarp0) {
      // ======================= bf16 -> fp16 conversion of V tiles (bf16 inputs) ======
      // Walks every ring item in order: waits for it to land, converts it if it is a V
      // tile, then arrives on its v_conv barrier (the MMA issuer waits on that for V
      // tiles) and on its empty barrier (the producer refills a stage only after both the
      // tensor core and the converters are done with it).
      // A V element of magnitude 65536 or more (or inf / NaN) has no fp16 value: the
      // largest magnitude bit pattern met is tracked per thread and, if any such element
      // was converted, the call's status word records kStatusRange.
      const int ct = threadIdx.x - C::kConvWarp0 * 32;  // 0..63
      uint32_t vmag = 0;  // per-halfword max of |bf16 bits| over every V element converted
      int g = 0;
      for (int k = 0;; ++k) {
        const Unit u = next_unit(k);
        if (u.nmax < 0) break;
        if constexpr (BF16) {
          for (int i = 0; i < 2 * u.nmax; ++i) {
            const int item = g + i;
            const int st = item % C::kStages;
            mbar_wait_inline(BAR(C::kBarKVFull + st), (item / C::kStages) & 1, wctx);
            __syncwarp();
            if (i & 1) {
              uint4* tile = reinterpret_cast<uint4*>(smem + C::kOffKV + st * C::kTileBytes);
#pragma unroll 4
              for (int c = ct; c < C::kTileBytes / 16; c += 64) {
                uint4 w = tile[c];
                vmag = __vmaxu2(vmag, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                               __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
                w.x = bf16x2_to_f16x2_sat(w.x);
                w.y = bf16x2_to_f16x2_sat(w.y);
                w.z = bf16x2_to_f16x2_sat(w.z);
                w.w = bf16x2_to_f16x2_sat(w.w);
                tile[c] = w;
              }
              fence_proxy_async_smem();  // generic-proxy writes -> visible to the tensor core
            }
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(BAR(C::kBarVConv + st));
              mbar_arrive(BAR(C::kBarKVEmpty + st));
            }
          }
        }
        g += 2 * u.nmax;
      }
      if (max(vmag & 0xFFFFu, vmag >> 16) >= kBf16NoF16) atomicCAS(p.status, 0, kStatusRange);
    }
    // back to the launch's registers (waits until the softmax warps have given theirs back)
    __syncwarp();
    if constexpr (C::kDecoupled) warpgroup_reg_alloc<C::kLaunchRegs>();
  } else {
    // warpgroups 0 and 1: softmax
    if constexpr (C::kDecoupled) warpgroup_reg_alloc<C::kRegsSoftmax>();
    if constexpr (C::kDecoupled) {
    // ======================= softmax warpgroups (warps 0-3: tile 0, 4-7: tile 1) ======
    const int t = warp >> 2;
    const int quarter = warp & 3;  // TMEM lane quarter this warp may access
    const int r = quarter * 32 + lane;  // row inside the Q tile
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_base + (t ? 128u : 0u);
    const uint32_t tO = tmem + lane_base + (t ? 256u + D : 256u);
    const uint32_t tP = tmem + lane_base + C::kColP + 64u * t;  // d = 64 only
    const float cs = p.scale_log2;
    const bool neg = cs < 0.f;
    const float cs_abs = fabsf(cs);
    uint8_t* ptile = smem + C::kOffO + t * C::kTileBytes;  // O staging of tile t
    int ns = 0;   // S tiles consumed (s_full phases)
    int njoin = 0;  // shared units joined
    int npv = 0;  // P V operations of this tile waited for (pv_done phases)
    int nout = 0;  // O tiles stored (o_free / o_ready phases)
    for (int k = 0;; ++k) {
      const Unit u = next_unit(k);
      if (u.nmax < 0) break;
      const int query = u.pos0[t] + (r >> p.lg_pack);  // this row's query and head
      const int head = u.h + (r & ((1 << p.lg_pack) - 1));
      if (u.end[u.shared() ? 0 : t] == 0) {
        // every row of this tile is left without a key (Nq > Nk): O = 0, lse = -inf
        if (query < p.Nq) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) +
                                                ((((long long)u.b * p.Nq + query) * p.H + head) * D) * 2);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
          if (p.lse != nullptr) p.lse[((long long)u.b * p.H + head) * p.Nq + query] = -INFINITY;
        }
        continue;
      }

      float m_run = -INFINITY;  // running max of scale*log2(e)*s (lazy: may lag the true max by <= 8)
      float l_run = 0.f;        // running sum of 2^(cs*s - m_run)
      const WindowRow row = window_row(p, u.pos0[t], query);
      for (int j = 0; j < u.end[t]; ++j) {
        if (!u.active(t, j)) continue;
        const bool first = u.starts(t, j);
        mbar_wait_inline(BAR(C::kBarSFull + t), ns & 1, wctx);
        ++ns;
        __syncwarp();  // lanes may leave the bounded wait on different polls
        tc_fence_after_sync();
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, sr[c]);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 4; ++c) reg_order_after_wait(sr[c]);
        // S_t is in registers: the tensor core may compute S_t(j+1) into the same columns
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::kBarSFree + t));

        // which of the tile's keys this row sees
        uint32_t see[4];
        const bool need_mask = row.masked(u, j, see);
        const float mx = need_mask ? (neg ? seen_row_max<true>(sr, see) : seen_row_max<false>(sr, see))
                                   : (neg ? row_max<false, true>(sr, 0) : row_max<false, false>(sr, 0));
        const float m_tile = (mx == -INFINITY) ? -INFINITY : mx * cs_abs;
        const float m_new = fmaxf(m_run, m_tile);
        const bool rescale = m_new > m_run + 8.0f;
        const float alpha = rescale ? ex2_approx(m_run - m_new) : 1.0f;
        if (rescale) {
          m_run = m_new;
          l_run *= alpha;
        }
        const float m_use = (m_run == -INFINITY) ? 0.f : m_run;

        if (!first) {
          // the previous P_t V must be done: its P buffer is about to be overwritten and O_t may be rescaled
          mbar_wait_inline(BAR(C::kBarPVDone + t), npv & 1, wctx);
          ++npv;
          __syncwarp();
          tc_fence_after_sync();
          if (__any_sync(0xffffffffu, rescale)) {  // lazy rescale of O (rare after the first tiles)
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_ld_wait();
              reg_order_after_wait(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(tO + c * 32, o);
            }
          }
        }

        l_run += need_mask ? window_row_exp_to_tmem<true>(sr, cs, m_use, see, tP)
                           : window_row_exp_to_tmem<false>(sr, cs, m_use, see, tP);
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::kBarPFull + t));
      }

      // ---- epilogue: O / l -> 16-bit -> swizzled staging (this tile's buffer) -> TMA store
      if (u.end[t] > 0) {
        mbar_wait_inline(BAR(C::kBarPVDone + t), npv & 1, wctx);
        ++npv;
      }
      __syncwarp();
      tc_fence_after_sync();
      if (u.shared() && t == 1) {  // slot 0's warps take it from here
        slot1[r] = make_float2(m_run, l_run);
        __syncwarp();
        if (lane == 0) mbar_arrive(join);
        mbar_wait_inline(join + 8, njoin++ & 1, wctx);
        __syncwarp();
        tc_fence_after_sync();
        continue;
      }
      float f1 = 0.f;
      const float inv_l = join_slots(u, slot1, r, m_run, l_run, f1, join, njoin, wctx);
      if (u.shared()) ++njoin;
      if (u.shared()) {
        // this tile's previous O store has read the staging buffer before it is rewritten
        if (r == 0) {
          bulk_wait_group_read0();
          mbar_arrive(BAR(C::kBarOFree + t));
        }
        mbar_wait_inline(BAR(C::kBarOFree + t), nout & 1, wctx);
        __syncwarp();
        stage_joined<D, BF16, kShared>(u, tO, tmem + lane_base + 256u + D, inv_l, f1, ptile, r, join);
      } else {
        uint32_t o[D / 32][32];  // the whole O row: one TMEM round trip
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tmem_ld32(tO + c * 32, o[c]);
        // this tile's previous O store has read the staging buffer before it is rewritten
        if (r == 0) {
          bulk_wait_group_read0();
          mbar_arrive(BAR(C::kBarOFree + t));
        }
        mbar_wait_inline(BAR(C::kBarOFree + t), nout & 1, wctx);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) reg_order_after_wait(o[c]);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {  // four 16-byte chunks of 8 elements
            uint4 w;
            w.x = pack2<BF16>(__uint_as_float(o[c][q4 * 8 + 0]) * inv_l, __uint_as_float(o[c][q4 * 8 + 1]) * inv_l);
            w.y = pack2<BF16>(__uint_as_float(o[c][q4 * 8 + 2]) * inv_l, __uint_as_float(o[c][q4 * 8 + 3]) * inv_l);
            w.z = pack2<BF16>(__uint_as_float(o[c][q4 * 8 + 4]) * inv_l, __uint_as_float(o[c][q4 * 8 + 5]) * inv_l);
            w.w = pack2<BF16>(__uint_as_float(o[c][q4 * 8 + 6]) * inv_l, __uint_as_float(o[c][q4 * 8 + 7]) * inv_l);
            const int chunk = c * 4 + q4;  // 16-byte chunk index along the row
            const int bx = chunk >> 3, cc = chunk & 7;
            *reinterpret_cast<uint4*>(ptile + bx * C::kBoxBytes + r * 128 + ((cc ^ (r & 7)) << 4)) = w;
          }
        }
      }
      fence_proxy_async_smem();  // generic-proxy writes -> visible to the TMA store
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::kBarOReady + t));
      if (quarter == 0) {
        mbar_wait_inline(BAR(C::kBarOReady + t), nout & 1, wctx);
        if (r == 0 && !*abort_flag) {
          for (int bx = 0; bx < C::kBoxes; ++bx)
            tma_store_4d(&p.tm_o, sbase + C::kOffO + t * C::kTileBytes + bx * C::kBoxBytes, bx * 64,
                         u.h, u.pos0[t], u.b);
          bulk_commit_group();
        }
      }
      ++nout;
      if (p.lse != nullptr && query < p.Nq) {
        const float lse = l_run > 0.f ? (m_run + lg2_approx(l_run)) * 0.69314718055994531f
                                      : -INFINITY;
        p.lse[((long long)u.b * p.H + head) * p.Nq + query] = lse;
      }
    }
    if (r == 0) bulk_wait_group_read0();  // the last O store has read the staging buffer
    } else {
    // ======================= softmax warpgroups (warps 0-3: tile 0, 4-7: tile 1) ======
    const int t = warp >> 2;
    const int quarter = warp & 3;  // TMEM lane quarter this warp may access
    const int r = quarter * 32 + lane;  // row inside the Q tile
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_base + (t ? 128u : 0u);
    const uint32_t tO = tmem + lane_base + (t ? 256u + D : 256u);
    const float cs = p.scale_log2;
    const bool neg = cs < 0.f;
    const float cs_abs = fabsf(cs);
    uint8_t* ostage = smem + C::kOffO;
    // The two tiles take turns with the one O staging buffer, in the order tile 0 of
    // unit 0, tile 1 of unit 0, tile 0 of unit 1, ...: a turn starts when the previous
    // turn's TMA store has finished reading the buffer (a tile without a store passes its turn).
    // Every warp of the slot arrives for its turn once it has seen the turn before end: were one
    // arrival enough, turns passed in a row could end a phase that a slower warp still waits for.
    auto ostage_acquire = [&](int k) {
      if (t == 0 && k > 0) mbar_wait_inline(BAR(C::kBarOStage + 1), (k - 1) & 1, wctx);
      if (t == 1) mbar_wait_inline(BAR(C::kBarOStage + 0), k & 1, wctx);
      __syncwarp();
    };
    int ns = 0;  // S tiles consumed (s_full phases)
    int odd = 0;  // bit 0: units finished are odd in number (o_full phases), bit 1: shared units joined are
    bool store_pending = false;  // (row 0's thread) this tile's last O store may still read the buffer
    for (int k = 0;; ++k) {
      const Unit u = next_unit(k);
      // The store issued at the end of the previous unit has had the unit switch to read
      // the staging buffer; only now does row 0's thread wait for it and pass the turn on.
      if (r == 0 && store_pending) {
        bulk_wait_group_read0();
        mbar_arrive(BAR(C::kBarOStage + t));
        store_pending = false;
      }
      if (u.nmax < 0) break;
      const int query = u.pos0[t] + (r >> p.lg_pack);  // this row's query and head
      const int head = u.h + (r & ((1 << p.lg_pack) - 1));
      if (u.end[u.shared() ? 0 : t] == 0) {
        ostage_acquire(k);  // pass this tile's turn with the staging buffer
        if (lane == 0) mbar_arrive(BAR(C::kBarOStage + t));
        // every row of this tile is left without a key (Nq > Nk): O = 0, lse = -inf
        if (query < p.Nq) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) +
                                                ((((long long)u.b * p.Nq + query) * p.H + head) * D) * 2);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
          if (p.lse != nullptr) p.lse[((long long)u.b * p.H + head) * p.Nq + query] = -INFINITY;
        }
        continue;
      }

      float m_run = -INFINITY;  // running max of scale*log2(e)*s (lazy: may lag the true max by <= 8)
      float l_run = 0.f;        // running sum of 2^(cs*s - m_run)
      const WindowRow row = window_row(p, u.pos0[t], query);
      for (int j = 0; j < u.end[t]; ++j) {
        if (!u.active(t, j)) continue;
        const bool first = u.starts(t, j);
        mbar_wait_inline(BAR(C::kBarSFull + t), ns & 1, wctx);
        ++ns;
        __syncwarp();  // lanes may leave the bounded wait on different polls
        tc_fence_after_sync();
        // which of the tile's keys this row sees
        uint32_t see[4];
        const bool need_mask = row.masked(u, j, see);

        // Speculative single pass: S read in two halves, exponentiated against m_run while
        // the tile max is found; P stays in registers and is written only if no exponent
        // exceeds 8 in any row of the warp (S is untouched until then), else the two-pass
        // path below redoes the tile.
        if (__all_sync(0xffffffffu, m_run != -INFINITY)) {
          uint32_t pk[2][32];
          float xmax = -INFINITY;
          float rs;
          {
            uint32_t sv[2][32];
            tmem_ld32(tS + 64, sv[0]);
            tmem_ld32(tS + 96, sv[1]);
            tmem_ld_wait();
            reg_order_after_wait(sv[0]);
            reg_order_after_wait(sv[1]);
            rs = need_mask ? window_half_exp<true, 1>(sv, cs, m_run, see, pk[1], xmax)
                           : window_half_exp<false, 1>(sv, cs, m_run, see, pk[1], xmax);
            tmem_ld32(tS + 0, sv[0]);
            tmem_ld32(tS + 32, sv[1]);
            tmem_ld_wait();
            reg_order_after_wait(sv[0]);
            reg_order_after_wait(sv[1]);
            rs += need_mask ? window_half_exp<true, 0>(sv, cs, m_run, see, pk[0], xmax)
                            : window_half_exp<false, 0>(sv, cs, m_run, see, pk[0], xmax);
          }
          if (!__any_sync(0xffffffffu, xmax > 8.0f)) {
            l_run += rs;
            tmem_st32(tS + 96, pk[1]);  // keys 64..127
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::kBarPHalf + t));
            tmem_st32(tS + 64, pk[0]);  // keys 0..63
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::kBarPFull + t));
            continue;
          }
        }

        // pass 1: row max over the two 64-column halves (half 1 stays in registers)
        uint32_t hv[2][32];
        tmem_ld32(tS + 0, hv[0]);
        tmem_ld32(tS + 32, hv[1]);
        tmem_ld_wait();
        reg_order_after_wait(hv[0]);
        reg_order_after_wait(hv[1]);
        float mx = need_mask ? (neg ? seen_half_max<true, 0>(hv, see) : seen_half_max<false, 0>(hv, see))
                             : (neg ? half_max<false, true, 0>(hv, 0) : half_max<false, false, 0>(hv, 0));
        tmem_ld32(tS + 64, hv[0]);
        tmem_ld32(tS + 96, hv[1]);
        tmem_ld_wait();
        reg_order_after_wait(hv[0]);
        reg_order_after_wait(hv[1]);
        mx = fmaxf(mx, need_mask ? (neg ? seen_half_max<true, 1>(hv, see) : seen_half_max<false, 1>(hv, see))
                                 : (neg ? half_max<false, true, 1>(hv, 0) : half_max<false, false, 1>(hv, 0)));
        const float m_tile = (mx == -INFINITY) ? -INFINITY : mx * cs_abs;
        const float m_new = fmaxf(m_run, m_tile);
        const bool rescale = m_new > m_run + 8.0f;
        const float alpha = rescale ? ex2_approx(m_run - m_new) : 1.0f;
        if (rescale) {
          m_run = m_new;
          l_run *= alpha;
        }
        const float m_use = (m_run == -INFINITY) ? 0.f : m_run;

        // lazy rescale of O, before any P_t(j) V_j can start (P_t(j-1) V_{j-1} completed
        // before S_t(j) did)
        if (!first && __any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + c * 32, o);
            tmem_ld_wait();
            reg_order_after_wait(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(tO + c * 32, o);
          }
        }

        // pass 2: P for half 1 (keys 64..127, from registers) into TMEM columns 96..127,
        // which held S columns 96..127 -- already read -- and published at once, so the
        // tensor core starts on keys 64..127 of P_t V_j; then half 0 re-read from TMEM
        // (columns 0..63, untouched) into P columns 64..95.
        uint32_t pk[32];
        float unused = -INFINITY;
        float rs = need_mask ? window_half_exp<true, 1>(hv, cs, m_use, see, pk, unused)
                             : window_half_exp<false, 1>(hv, cs, m_use, see, pk, unused);
        __syncwarp();
        tmem_st32(tS + 96, pk);
        tmem_ld32(tS + 0, hv[0]);
        tmem_ld32(tS + 32, hv[1]);
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::kBarPHalf + t));
        tmem_ld_wait();
        reg_order_after_wait(hv[0]);
        reg_order_after_wait(hv[1]);
        rs += need_mask ? window_half_exp<true, 0>(hv, cs, m_use, see, pk, unused)
                        : window_half_exp<false, 0>(hv, cs, m_use, see, pk, unused);
        l_run += rs;
        __syncwarp();
        tmem_st32(tS + 64, pk);
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::kBarPFull + t));
      }

      // ---- epilogue: O / l -> 16-bit -> swizzled staging buffer -> TMA store
      if (u.end[t] > 0) {
        mbar_wait_inline(BAR(C::kBarPVDone + t), odd & 1, wctx);
        odd ^= 1;
      }
      __syncwarp();
      tc_fence_after_sync();
      if (u.shared() && t == 1) {  // slot 0's warps take it from here
        slot1[r] = make_float2(m_run, l_run);
        __syncwarp();
        if (lane == 0) mbar_arrive(join);
        // Slot 0's turn with the staging buffer is over: O_1 and slot1 have been read.  Pass slot 1's.
        ostage_acquire(k);
        if (lane == 0) mbar_arrive(BAR(C::kBarOStage + 1));
        continue;
      }
      float f1 = 0.f;
      const float inv_l = join_slots(u, slot1, r, m_run, l_run, f1, join, odd >> 1, wctx);
      if (u.shared()) odd ^= 2;
      ostage_acquire(k);  // the previous store from the staging buffer has read it
      if (u.shared()) {
        stage_joined<D, BF16, kShared>(u, tO, tmem + lane_base + 256u + D, inv_l, f1, ostage, r, join);
      } else {
        uint32_t o[D / 32][32];  // the whole O row: one TMEM round trip
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tmem_ld32(tO + c * 32, o[c]);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) reg_order_after_wait(o[c]);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {  // four 16-byte chunks of 8 elements
            uint4 w;
            w.x = pack2<BF16>(__uint_as_float(o[c][q4 * 8 + 0]) * inv_l, __uint_as_float(o[c][q4 * 8 + 1]) * inv_l);
            w.y = pack2<BF16>(__uint_as_float(o[c][q4 * 8 + 2]) * inv_l, __uint_as_float(o[c][q4 * 8 + 3]) * inv_l);
            w.z = pack2<BF16>(__uint_as_float(o[c][q4 * 8 + 4]) * inv_l, __uint_as_float(o[c][q4 * 8 + 5]) * inv_l);
            w.w = pack2<BF16>(__uint_as_float(o[c][q4 * 8 + 6]) * inv_l, __uint_as_float(o[c][q4 * 8 + 7]) * inv_l);
            const int chunk = c * 4 + q4;  // 16-byte chunk index along the row
            const int bx = chunk >> 3, cc = chunk & 7;
            *reinterpret_cast<uint4*>(ostage + bx * C::kBoxBytes + r * 128 + ((cc ^ (r & 7)) << 4)) = w;
          }
        }
      }
      fence_proxy_async_smem();  // generic-proxy writes -> visible to the TMA store
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::kBarOReady + t));
      if (lane == 0 && quarter != 0) mbar_arrive(BAR(C::kBarOStage + t));
      if (quarter == 0) {
        mbar_wait_inline(BAR(C::kBarOReady + t), (odd & 1) ^ 1, wctx);
        if (r == 0 && !*abort_flag) {
          for (int bx = 0; bx < C::kBoxes; ++bx)
            tma_store_4d(&p.tm_o, sbase + C::kOffO + bx * C::kBoxBytes, bx * 64, u.h, u.pos0[t], u.b);
          bulk_commit_group();
        }
      }
      store_pending = true;  // completed (and the turn passed on) after the next unit is read
      if (p.lse != nullptr && query < p.Nq) {
        const float lse = l_run > 0.f ? (m_run + lg2_approx(l_run)) * 0.69314718055994531f
                                      : -INFINITY;
        p.lse[((long long)u.b * p.H + head) * p.Nq + query] = lse;
      }
    }
    }
    __syncwarp();
    if constexpr (C::kDecoupled) warpgroup_reg_dealloc<C::kLaunchRegs>();
  }

  // ---- teardown: every role is done with TMEM
  tc_fence_before_sync();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace attn_b200
