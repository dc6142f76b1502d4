// split_sm100.cuh -- attention of a few query rows over many keys, split over the keys: one
// token (or a few) of grouped heads against a dense 16-bit K/V or the paged 4-bit cache of
// q4_cache.cuh, with an optional window and sinks (sm_100a).
//
// The rows of a (request, key/value head) are its Lq tokens of G heads; 8 NT of them make an
// item.  Every key and value is read once per item and used by all its rows, so the step is
// bound by the read of the cache; tcgen05's 128-row tiles would stay empty, and mma.sync
// (16 keys x 8 rows) takes the products:
//   S^T = K Q^T (A = 16 keys x 16 channels),   O^T += V^T P^T (A = 16 channels x 16 keys);
// S^T and O^T hold a key's or channel's row and two query columns per thread, so the running
// maximum, sum and rescale of a query stay in a thread, and P^T becomes the second product's
// operand by one 8x8 transposition (movmatrix).
//
// 4-bit codes multiply as they are, with no conversion to values: a code c at bit 0 or 4 of a
// 16-bit half is the fp16 subnormal c 2^-24 or c 2^-20, exact on the tensor cores, so a logic
// instruction (and a shift for every second) makes an operand of two codes.
//   K: a group of 64 channels adds 2^24 s acc + z sum q to the score, acc the fp32 product.  q
//      enters scaled by a power of two to [2^14, 2^15) at its row's largest element, and by 1/16
//      in the channels whose codes lie at bit 4: exact, for bf16 rows too, down to 2^-25 of that
//      element (and off by 2^-36 of it below);
//   V: codes multiply P' = p s / R rounded to fp16.  R is a power of two at or above the group's
//      largest scale so far, so P' keeps 11 bits where p s lies within 2^-14 of R.  Codes are
//      counted from their middle 8 (8 R sum P' is taken off, over the rounded P'), so that
//      rounding P' costs what rounding p against the values would, or twice that where a group's
//      zero is off its middle; sum P' is one more product, with ones, and sum p (z + 8 s) is
//      fp32.  fp16 outputs, which would show it (3.8e-4 of the result against 2.1e-4 for a
//      rounding of the exact one), take P' as the sum of two fp16 values instead, a product each.
//
// Work: an item's keys are a stream of chunks of 16 KT keys.  The chunks of all items, end to
// end, are dealt to the CTAs in equal runs (each CTA finds its run from the lengths), so ragged
// requests keep every SM busy to the end; a run's whole items are finished by its CTA, the parts
// of split ones go to a workspace, and the CTA that comes last puts an item's together, in key
// order.  (A second launch for that cost 6 us.)  Where the items are few enough and not too uneven
// (split_parts), each is cut into as many equal parts as there are CTAs for it instead, so that a
// CTA has one part: a part costs about 5 us besides its chunks.  Calls whose items are all
// short take one CTA an item and no workspace.
// A warp works alone on every 8th chunk of a run: its lanes start bulk (4-bit) or tiled (16-bit)
// copies into its own ring of stages and wait on its own barriers; the warps' partial rows meet
// in shared memory at the end of an item's part.
#pragma once

#include <type_traits>

#include "prefill_sm100.cuh"  // bounded waits without a call
#include "q4_cache.cuh"

namespace attn_b200 {

struct SplitParams {
  CUtensorMap tm_k;   // dense: k [B, Nk, Hkv, D] as (D, Hkv, Nk, B), box (64, 1, 16, 1), 128B swizzle
  CUtensorMap tm_v;   // same
  const uint8_t* cache;    // 4-bit: the cache, its table and lengths
  const int* block_table;
  const int* seq_lens;
  const void* q;      // [B, Lq, H, D]
  void* out;          // [B, Lq, H, D]
  float* lse;         // [B, H, Lq] or nullptr
  int* status;
  int B, H, Hkv, Lq;
  int Nk;             // dense: keys; 4-bit: max_blocks * page_size
  int causal, window, sinks;
  int num_blocks, page_size, max_blocks;
  int row_chunks;     // items per (request, key/value head)
  float* part;        // nullptr: one CTA an item.  Else [2 CTAs][kRows][D + 4]: o, maximum, sum
  unsigned long long* arrived;  // [CTAs]: parts of the item whose first one is the CTA's (see split_arrive)
  unsigned long long nonce;     // of the launch, its low 16 bits 0
  float scale_log2;
  unsigned long long timeout_ns;
  int inject;         // test hook: 1 = the first chunk of each CTA never counts as landed
};

template <int D, bool Q4, int NT>
struct SplitCfg {
  static constexpr int kWarps = 8;
  static constexpr int kRows = 8 * NT;                        // query rows of an item
  static constexpr int kTiles = (Q4 && NT < 4) ? 2 : 1;       // 16-key tiles of a chunk
  static constexpr int kMinRun = 2 * kWarps;                  // chunks of a CTA, where there are fewer than for all
  static constexpr int kTileBytes = Q4 ? 16 * (9 * D / 8) : 16 * D * 4;
  static constexpr int kStageBytes = kTiles * kTileBytes;
  static constexpr int kStages = 3;
  static constexpr int kPitch = D + 4;                        // floats of a partial row
  static constexpr int kPartBytes = kRows * kPitch * 4;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  // the partials of the warps lie over the ring once a part of an item is done
  static constexpr int kOverlay = kWarps * kPartBytes;
  static constexpr int kOffQ = ((kRingBytes > kOverlay ? kRingBytes : kOverlay) + 127) / 128 * 128;
  static constexpr int kQBytes = (D / 16) * NT * 32 * 8;      // Q as the products' B operands
  static constexpr int kOffSum = kOffQ + kQBytes;             // float [D / 64 + 1][kRows]: sums of q, scale of a row
  static constexpr int kOffMl = kOffSum + (D / 64 + 1) * kRows * 4;  // float [kWarps][kRows][2]: maximum, sum
  static constexpr int kOffBar = kOffMl + kWarps * kRows * 8;
  static constexpr int kOffAbort = kOffBar + kWarps * kStages * 8;
  static constexpr int kSmemBytes = kOffAbort + 16 + 1024;    // +1024: manual 1 KB alignment
  static constexpr int kCtas = (NT == 1 && kSmemBytes <= 113 * 1024) ? 2 : 1;  // resident on an SM
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
               : "memory");
}

// D (16 x 8, fp32) = A (16 x 16) B (16 x 8) + C
template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
  if constexpr (BF16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  }
}
// D += A B, or D = A B
template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1, bool fresh = false) {
  if (fresh) mma_16816<BF16>(d, a0, a1, a2, a3, b0, b1, 0.f, 0.f, 0.f, 0.f);
  else mma_16816<BF16>(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <bool kTrans>
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  if constexpr (kTrans)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ float group_max(float x) {  // over the 8 lanes that share lane % 4
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// What the rows of request b see: keys [low, len) and the sinks, as a stream of 16-key tiles
// (those of the sinks that lie before the window's, then the window's).
struct SplitSpan {
  int len, low, first, n_sink, n_tiles;
  __device__ __forceinline__ int tile_key(int x) const { return 16 * (x < n_sink ? x : first + x - n_sink); }
};

// First key of the window of a row at position pos.
__device__ __forceinline__ int split_edge(const SplitParams& p, int pos) {
  return p.window > 0 ? (int)max(0LL, (long long)pos - p.window + 1) : 0;
}

template <bool Q4>
__device__ __forceinline__ SplitSpan split_span(const SplitParams& p, int b) {
  SplitSpan s;
  s.len = Q4 ? min(max(__ldg(p.seq_lens + b), 0), p.Nk) : p.Nk;
  s.low = split_edge(p, p.causal ? max(s.len - p.Lq, 0) : s.len - 1);
  s.first = s.low / 16;
  s.n_sink = p.window > 0 ? min((int)(((long long)min(p.sinks, p.Nk) + 15) / 16), s.first) : 0;
  s.n_tiles = s.len > 0 ? s.n_sink + (s.len - 1) / 16 - s.first + 1 : 0;
  return s;
}

// Place in the chunks of all items end to end (requests, then their items): a chunk of request b,
// whose first item begins at `begin`.
struct SplitPlace {
  int b;
  long long begin;
};

template <int D, bool Q4, int NT>
__device__ __forceinline__ int split_chunks(const SplitParams& p, int b) {  // of an item of request b
  constexpr int kTiles = SplitCfg<D, Q4, NT>::kTiles;
  return b < p.B ? (split_span<Q4>(p, b).n_tiles + kTiles - 1) / kTiles : 0;
}

// Number of chunks of all items, and of the longest item (a whole warp together).
template <int D, bool Q4, int NT>
__device__ __forceinline__ long long split_total(const SplitParams& p, int& longest) {
  long long total = 0;
  longest = 0;
  for (int b = threadIdx.x & 31; b < p.B; b += 32) {
    const int n = split_chunks<D, Q4, NT>(p, b);
    total += n;
    longest = max(longest, n);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
  }
  return total * p.Hkv * p.row_chunks;
}

// The place of chunk x (a whole warp together).
template <int D, bool Q4, int NT>
__device__ __forceinline__ SplitPlace split_find(const SplitParams& p, long long x) {
  const int lane = threadIdx.x & 31;
  const long long per = (long long)p.Hkv * p.row_chunks;
  long long begin = 0;
  SplitPlace place{p.B, 0};
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int c = split_chunks<D, Q4, NT>(p, b0 + lane);
    const long long n = c * per;
    long long sum = n;  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    const unsigned past = __ballot_sync(0xffffffffu, begin + sum > x);
    if (past != 0) {
      const int l = __ffs(past) - 1;
      place.b = b0 + l;
      place.begin = begin + __shfl_sync(0xffffffffu, sum - n, l);
      break;
    }
    begin += __shfl_sync(0xffffffffu, sum, 31);
  }
  return place;
}

// Chunks of a CTA's run (the last may be shorter).
__device__ __forceinline__ long long split_run(long long total, int grid, int min_run) {
  return max((long long)min_run, (total + grid - 1) / grid);
}

// Parts that each item is cut into, one a CTA, or 0: runs of equal length instead.  The longest
// part is the time of the first, chunks and about 5 us for a part; a CTA of the second has up to an
// equal share of all chunks, but two or three parts.  So parts pay up to some chunks more than that share:
// with 4 min_run (64) of them, one token over the cache, 32 heads over 8, 8 requests of 1500 to 3000
// keys take 23.1 us against 30.4 in runs, 34 of 4500 to 6000 70.6 against 77.9; 16 of 40000 take
// 187.8 in runs against 198.7 in parts.  Chunks of other items, with 0, 4 and 16 min_run (inputs not in
// L2): 4-bit, 8 requests of 1500 to 3000 keys, 16 rows 33.4 27.2 27.2, 32 rows 53.9 45.7 45.7; 5 of 500 to
// 20000, 16 rows 49.8 49.8 55.9, 32 rows 94.8 94.8 115.3; 12 of 3000 to 9000, 16 rows 45.7 47.7 66.1; dense,
// 4096 keys, 5 requests, 4 rows 33.4 31.3 29.3, 16 rows 39.5 33.4 35.4; 16 requests 64.1 62.0 62.0 and 70.2
// 66.1 66.1.
__device__ __forceinline__ int split_parts(long long total, int longest, long long items, int grid, int min_run) {
  const int most = (int)(grid / items);
  if (most == 0) return 0;
  const int parts = max(1, min(most, longest / min_run));
  return (longest + parts - 1) / parts <= split_run(total, grid, min_run) + 4 * min_run ? parts : 0;
}

// Running maximum of a row that has seen no key: finite, so that differences from it are.
constexpr float kNoMax = -1e30f;

// Counts a part of an item in; true for the last of n.  The word comes from a memory pool with
// anything in it: a count is one only under the launch's nonce (48 random bits, so that a word
// left by others passes for it once in 2^48), and the last part clears the word, so that a
// replayed launch with the same nonce starts afresh.  So every part is counted in, those of a CTA
// that gives up too: a count left behind would make the replay take an early part for the last.
// (To count them in without the parts' loop took registers: 16 requests of 8000 to 16000 keys 112 ->
// 114 us.)
__device__ __forceinline__ bool split_arrive(unsigned long long* word, unsigned long long nonce, int n) {
  // the last part's guess is right at once, the others' time does not count
  unsigned long long seen = nonce | (unsigned long long)(n - 1);
  while (true) {
    const unsigned long long count = ((seen ^ nonce) >> 16) == 0 ? (seen & 0xffffu) + 1 : 1;
    const bool last = count == (unsigned long long)n;
    const unsigned long long was = atomicCAS(word, seen, last ? 0ull : nonce | count);
    if (was == seen) return last;
    seen = was;
  }
}

// Four channels of the sum of partial rows: o and l in units of 2^m, m the largest of their maxima.
struct SplitSum {
  float4 o;
  float m, l;
};

// The same for a fixed number of partials, their weights side by side.
template <int n, typename ML, typename O>
__device__ __forceinline__ SplitSum split_sum_fixed(ML&& load_ml, O&& load_o) {
  float2 w[n];
#pragma unroll
  for (int i = 0; i < n; ++i) w[i] = load_ml(i);
  SplitSum a{make_float4(0.f, 0.f, 0.f, 0.f), kNoMax, 0.f};
#pragma unroll
  for (int i = 0; i < n; ++i) a.m = fmaxf(a.m, w[i].x);
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const float f = ex2_approx(w[i].x - a.m);
    const float4 v = load_o(i);
    a.l = fmaf(f, w[i].y, a.l);
    a.o.x = fmaf(f, v.x, a.o.x);
    a.o.y = fmaf(f, v.y, a.o.y);
    a.o.z = fmaf(f, v.z, a.o.z);
    a.o.w = fmaf(f, v.w, a.o.w);
  }
  return a;
}

template <typename ML, typename O>
__device__ __forceinline__ SplitSum split_sum(int n, ML&& load_ml, O&& load_o) {
  SplitSum a{make_float4(0.f, 0.f, 0.f, 0.f), kNoMax, 0.f};
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float2 w = load_ml(i);
    const float4 v = load_o(i);
    const float top = fmaxf(a.m, w.x);
    const float e = ex2_approx(a.m - top), f = ex2_approx(w.x - top);  // 1 and the other's weight
    a.m = top;
    a.l = fmaf(f, w.y, e * a.l);
    a.o.x = fmaf(f, v.x, e * a.o.x);
    a.o.y = fmaf(f, v.y, e * a.o.y);
    a.o.z = fmaf(f, v.z, e * a.o.z);
    a.o.w = fmaf(f, v.w, e * a.o.w);
  }
  return a;
}

// Row r (of the rows of request b and key/value head hk) in q and out, in elements.
__device__ __forceinline__ long long split_row(const SplitParams& p, int b, int hk, int r, int G, int D) {
  return (((long long)b * p.Lq + r / G) * p.H + hk * G + r % G) * D;
}

template <int D, bool BF16>
__device__ __forceinline__ void split_store(const SplitParams& p, int b, int hk, int r, int c4, const SplitSum& a) {
  const int G = p.H / p.Hkv;
  const float inv = a.l > 0.f ? 1.0f / a.l : 0.f;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + split_row(p, b, hk, r, G, D) + c4) =
      make_uint2(pack2<BF16>(a.o.x * inv, a.o.y * inv), pack2<BF16>(a.o.z * inv, a.o.w * inv));
  if (c4 == 0 && p.lse != nullptr)
    p.lse[((long long)b * p.H + hk * G + r % G) * p.Lq + r / G] =
        a.l > 0.f ? (a.m + lg2_approx(a.l)) * 0.69314718055994531f : -INFINITY;
}

template <int D, bool BF16, bool Q4, int NT>
__global__ void __launch_bounds__(256, SplitCfg<D, Q4, NT>::kCtas)
    attn_split_kernel(const __grid_constant__ SplitParams p) {
  using C = SplitCfg<D, Q4, NT>;
  constexpr int kGroups = D / 64;
  constexpr int kM = D / 16;  // channel tiles of the output
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t sbase = (raw_addr + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw_addr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffAbort);
  volatile int* last_part = abort_flag + 1;
  const WaitCtx wctx{abort_flag, p.status, p.timeout_ns};

  const int G = p.H / p.Hkv;
  const int sinks = min(p.sinks, p.Nk);

  // ---- this warp's ring
  const uint32_t ring = sbase + warp * C::kStages * C::kStageBytes;
  const uint32_t bars = sbase + C::kOffBar + warp * C::kStages * 8;
  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(bars + 8 * s, p.inject == 1 && warp == 0 && s == 0 ? 2 : 1);
    mbar_init_fence();
  }
  if (threadIdx.x == 0) *abort_flag = 0;
  __syncthreads();

  const int T = Q4 ? min(p.page_size, kQ4MaxTile) : 16;  // tokens of a cache tile
  const int lg_pieces = (C::kTiles == 2 ? 1 : 0) + (T == 8 ? 1 : 0);  // log2 of the cache tiles of a chunk
  const int pieces = 1 << lg_pieces;
  const int piece_bytes = T * (9 * D / 8);
  const int per_load = 32 >> lg_pieces;

  // ---- the run of chunks of this CTA
  long long run = 0, run_end = 0, run_length = 1;
  int parts = 0;  // of an item (split_parts)
  SplitPlace place{(int)(blockIdx.x / (p.Hkv * p.row_chunks)), 0};
  if (p.part != nullptr) {
    // rows of requests without keys, dealt to the CTAs in turn
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
      if (split_span<Q4>(p, b).n_tiles > 0) continue;
      uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (long long)b * p.Lq * p.H * D);
      const long long rows = (long long)p.Lq * p.H;  // below 2^31, their elements are not
      for (long long e = threadIdx.x; e < rows * (D / 4); e += 256) dst[e] = make_uint2(0u, 0u);
      if (p.lse != nullptr)
        for (long long e = threadIdx.x; e < rows; e += 256) p.lse[(long long)b * p.H * p.Lq + e] = -INFINITY;
    }
    int longest;
    const long long total = split_total<D, Q4, NT>(p, longest);
    const int per = p.Hkv * p.row_chunks;
    parts = split_parts(total, longest, (long long)p.B * per, gridDim.x, C::kMinRun);
    if (parts > 0) {
      if (blockIdx.x >= (long long)p.B * per * parts) return;
      place.b = (int)(blockIdx.x / parts) / per;
    } else {
      run_length = split_run(total, gridDim.x, C::kMinRun);
      run = run_length * blockIdx.x;
      run_end = min(total, run + run_length);
      if (run >= run_end) return;
      place = split_find<D, Q4, NT>(p, run);
    }
  }
  int st = 0;          // the ring's stage of the warp's next chunk, and
  uint32_t phase = 0;  // its barrier's parity

  // ---- the parts of items in the run
  while (true) {
    const int b = place.b;
    const SplitSpan span = split_span<Q4>(p, b);
    const int n_chunks = (span.n_tiles + C::kTiles - 1) / C::kTiles;  // of the item
    int item, ca, cb;                                                 // item of the request, chunks [ca, cb) of it
    if (p.part == nullptr) {
      item = blockIdx.x % (p.Hkv * p.row_chunks);
      ca = 0;
      cb = n_chunks;
    } else if (parts > 0) {
      item = (int)(blockIdx.x / parts) % (p.Hkv * p.row_chunks);
      const int length = (n_chunks + parts - 1) / parts;
      ca = (int)(blockIdx.x % parts) * length;
      cb = min(n_chunks, ca + length);
      if (ca >= cb) return;
    } else {
      item = (int)((run - place.begin) / n_chunks);
      ca = (int)(run - place.begin - (long long)item * n_chunks);
      cb = (int)min((long long)n_chunks, ca + run_end - run);
    }
    const int hk = item / p.row_chunks;
    const int chunk_row0 = (item - hk * p.row_chunks) * C::kRows;
    const int rows = min(C::kRows, p.Lq * G - chunk_row0);  // rows of this item
    const int len = span.len;
    auto position = [&](int r) -> int {  // of the item's row r
      return p.causal ? len - p.Lq + (chunk_row0 + r) / G : len - 1;
    };
    const int pos_min = position(0), pos_max = position(rows - 1);
    const int low = split_edge(p, max(pos_min, 0)), low_max = split_edge(p, max(pos_max, 0));
    // stream tiles that every row sees whole: [0, sinks_end) and [all_from, all_end)
    const int sinks_end = min(span.n_sink, sinks / 16);
    const int all_from = span.n_sink + (low_max + 15) / 16 - span.first;
    const int all_end = span.n_sink + (pos_min + 1) / 16 - span.first;
    const int c0 = ca + warp;
    // chunks of this warp; none once the CTA has given up, whose parts are still counted in (split_arrive)
    const int mine = cb > c0 && !warp_flag(abort_flag) ? (cb - c0 + C::kWarps - 1) / C::kWarps : 0;

    // lane l: cache tile l % pieces of the warp's chunk (k / per_load) * per_load + l / pieces
    const uint8_t* piece = nullptr;
    unsigned have = 0;  // lanes with a cache tile
    auto issue = [&](int k, int at) {  // copies of this warp's k-th chunk of the part into stage `at`
      const uint32_t bar = bars + 8 * at;
      const uint32_t dst = ring + at * C::kStageBytes;
      if constexpr (Q4) {
        const int slot = k & (per_load - 1);
        if (slot == 0) {
          const int off = (lane & (pieces - 1)) * T;  // key within the chunk
          const int x = (c0 + (k + (lane >> lg_pieces)) * C::kWarps) * C::kTiles + off / 16;
          const int key = span.tile_key(x) + off % 16;
          const bool valid = k + (lane >> lg_pieces) < mine && x < span.n_tiles && key < len;
          have = __ballot_sync(0xffffffffu, valid);
          if (valid) {
            const int page = key / p.page_size;
            const int block = __ldg(p.block_table + (long long)b * p.max_blocks + page);
            piece = p.cache + q4_place<D>(min(max(block, 0), p.num_blocks - 1), hk, key - page * p.page_size, p.Hkv,
                                          p.page_size).tile;
          }
        }
        const unsigned these = (have >> (slot << lg_pieces)) & ((1u << pieces) - 1u);
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(these) * piece_bytes);
        __syncwarp();
        if ((lane >> lg_pieces) == slot && ((have >> lane) & 1u))
          bulk_load(dst + (lane & (pieces - 1)) * piece_bytes, piece, piece_bytes, bar);
      } else {
        if (lane == 0) mbar_arrive_expect_tx(bar, C::kStageBytes);
        __syncwarp();
        if (lane < 2 * kGroups) {  // K boxes, then V boxes; rows past Nk arrive as zeros
          const int bx = lane % kGroups;
          tma_load_4d(dst + lane * 2048, lane < kGroups ? &p.tm_k : &p.tm_v, bar, bx * 64, hk,
                      span.tile_key((c0 + k * C::kWarps) * C::kTiles), b);
        }
      }
      __syncwarp();
    };
    constexpr int kQWords = D / 64, kQRows = (C::kRows + C::kWarps - 1) / C::kWarps;
    [[maybe_unused]] uint32_t qw[kQRows][kQWords];  // 4-bit: this warp's rows of q, under way while the copies start
    if constexpr (Q4) {
#pragma unroll
      for (int i = 0; i < kQRows; ++i)
#pragma unroll
        for (int e = 0; e < kQWords; ++e) {
          const int row = warp + i * C::kWarps;
          qw[i][e] = row < rows ? __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.q) +
                                                                          split_row(p, b, hk, chunk_row0 + row, G, D)) +
                                        lane * kQWords + e)
                                : 0u;
        }
    }
    for (int k = 0; k < min(mine, C::kStages); ++k) issue(k, st + k < C::kStages ? st + k : st + k - C::kStages);

    // ---- Q as B operands; 4-bit: scaled to fp16 row by row, with its sums over 64 channels
    uint2* qf = reinterpret_cast<uint2*>(smem + C::kOffQ);      // [D / 16][NT][32]
    float* qsum = reinterpret_cast<float*>(smem + C::kOffSum);  // [kGroups][kRows], then the rows' scales
    const uint16_t* q = static_cast<const uint16_t*>(p.q);
    if constexpr (Q4) {
      uint16_t* qh = reinterpret_cast<uint16_t*>(smem + C::kOffQ);
#pragma unroll
      for (int i = 0; i < kQRows; ++i) {
        const int r = warp + i * C::kWarps;
        constexpr int E = D / 32;
        float x[E], s = 0.f, big = 0.f;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 f = unpack2<BF16>(qw[i][e / 2]);
          x[e] = f.x;
          x[e + 1] = f.y;
          s += f.x + f.y;
          big = fmax3(big, fabsf(f.x), fabsf(f.y));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
#pragma unroll
        for (int o = 16 / kGroups; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        // 2^(14 - exponent of the largest), kept where it and its inverse are normal numbers
        const int ex = max((int)(__float_as_uint(big) >> 23), 15);
        float up = __uint_as_float((uint32_t)(268 - ex) << 23);
        // a score is `unit` times what the products come to; masked ones are -inf in both
        const float unit = __uint_as_float((uint32_t)(ex - 14) << 23) * 16777216.f * fabsf(p.scale_log2);
        if (p.scale_log2 < 0.f) up = -up;
        if (lane % (32 / kGroups) == 0) qsum[(lane * kGroups / 32) * C::kRows + r] = s * up * 5.9604645e-8f;
        if (lane == 0) qsum[kGroups * C::kRows + r] = fmaxf(unit, 1e-37f);
        // channel ch of a group is the operand of lane 4 (r % 8) + ch / 16, step ch % 4
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int c = lane * E + e, ch = c % 64;
          const int at = ((c / 64 * 4 + ch % 4) * NT + r / 8) * 32 + (r % 8) * 4 + ch / 16;
          qh[at * 4 + ch % 16 / 4] = __half_as_ushort(__float2half_rn(x[e] * ((ch & 1) ? 0.0625f * up : up)));
        }
      }
    } else {
      for (int e = threadIdx.x; e < (D / 16) * NT * 32; e += 256) {
        const int el = e & 31, ks = e / 32 / NT, row = (e / 32 % NT) * 8 + (el >> 2);
        uint2 w = make_uint2(0u, 0u);
        if (row < rows) {
          const uint16_t* src = q + split_row(p, b, hk, chunk_row0 + row, G, D) + ks * 16 + (el & 3) * 2;
          w = make_uint2(*reinterpret_cast<const uint32_t*>(src), *reinterpret_cast<const uint32_t*>(src + 8));
        }
        qf[e] = w;
      }
    }
    __syncthreads();

    float qs[kGroups][NT][2] = {}, unit[NT][2];
    int pos[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = nt * 8 + 2 * t + c;
        pos[nt][c] = position(min(r, rows - 1));
        if constexpr (Q4) {
          unit[nt][c] = qsum[kGroups * C::kRows + r];
#pragma unroll
          for (int gg = 0; gg < kGroups; ++gg) qs[gg][nt][c] = qsum[gg * C::kRows + r];
        } else {
          unit[nt][c] = 1.f;
        }
      }

    float o[kM][NT][4] = {};
    float m[NT][2], l[NT][2] = {};
    float csum[kGroups][NT][4] = {}, zsum[kGroups][NT][2] = {};  // 4-bit: sums of P' and of p (z + 8 s)
    float big[kGroups], inv_big[kGroups];                        // 4-bit: R and 1 / R
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = kNoMax;
#pragma unroll
    for (int gg = 0; gg < kGroups; ++gg) {
      big[gg] = 5.9604645e-8f;  // 2^-24, the smallest scale there is
      inv_big[gg] = 16777216.f;
    }

    // the rows of a chunk: S^T's rows g and g + 8 are keys row_a and row_a + 8.  4-bit tiles take
    // them in an order that spreads the V rows of a word's load over the banks.
    const int row_a = Q4 ? (g >> 1) + 4 * (g & 1) : g;
    // byte offsets of a lane's reads within a 16-key tile (cache tiles of T tokens back to back)
    auto in_tile = [&](int row, int off) -> int {  // off: of the row 0 of a cache tile
      return row / T * piece_bytes + off;
    };
    int off_k[2], off_par[2], off_v[4];
    if constexpr (Q4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = row_a + 8 * i;
        off_k[i] = in_tile(row, row % T * (D / 2) + t * 8);
        off_par[i] = in_tile(row, T * D + row % T * (D / 8));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // keys of columns 2t, 2t + 1, 2t + 8, 2t + 9 of the A operand
        const int row = t + 4 * (i & 1) + 8 * (i >> 1);
        off_v[i] = in_tile(row, (T + row % T) * (D / 2) + g * 4);
      }
    }

    int k = 0;
    for (; k < mine; ++k) {
      const bool landed = mbar_wait_inline(bars + 8 * st, phase, wctx);
      if (!__all_sync(0xffffffffu, landed)) break;
      const uint8_t* stage = smem + warp * C::kStages * C::kStageBytes + st * C::kStageBytes;
      const uint32_t stage_addr = ring + st * C::kStageBytes;
      const int x0 = (c0 + k * C::kWarps) * C::kTiles;

      // ---- scores: base-2 exponents are unit times s
      float s[C::kTiles][NT][4];
      // parameters of this thread's two keys of a tile (K's or V's), as they are stored
      auto params = [&](int i, int h, int which, uint32_t (&w)[kGroups]) {
        const uint8_t* src = stage + i * C::kTileBytes + off_par[h] + which * (4 * kGroups);
        if constexpr (D == 128) {
          const uint2 v = *reinterpret_cast<const uint2*>(src);
          w[0] = v.x;
          w[1] = v.y;
        } else {
          w[0] = *reinterpret_cast<const uint32_t*>(src);
        }
      };
      if constexpr (Q4) {
        uint32_t par[C::kTiles][2][kGroups];
#pragma unroll
        for (int i = 0; i < C::kTiles; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) params(i, h, 0, par[i][h]);
#pragma unroll
        for (int gg = 0; gg < kGroups; ++gg) {
          float acc[C::kTiles][NT][4];
          uint2 w[C::kTiles][2];
#pragma unroll
          for (int i = 0; i < C::kTiles; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              w[i][h] = *reinterpret_cast<const uint2*>(stage + i * C::kTileBytes + off_k[h] + gg * 32);
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            uint2 bq[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) bq[nt] = qf[((gg * 4 + n) * NT + nt) * 32 + lane];
            const uint32_t mask = (n & 1) ? 0x00F000F0u : 0x000F000Fu;
#pragma unroll
            for (int i = 0; i < C::kTiles; ++i) {
              if (n == 2) {
                w[i][0].x >>= 8; w[i][0].y >>= 8; w[i][1].x >>= 8; w[i][1].y >>= 8;
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_16816<false>(acc[i][nt], w[i][0].x & mask, w[i][1].x & mask, w[i][0].y & mask, w[i][1].y & mask, bq[nt].x,
                                 bq[nt].y, n == 0);
            }
          }
#pragma unroll
          for (int i = 0; i < C::kTiles; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float2 sz = unpack2<false>(par[i][h][gg]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  float& x = s[i][nt][2 * h + c];
                  const float zq = gg == 0 ? sz.y * qs[gg][nt][c] : fmaf(sz.y, qs[gg][nt][c], x);
                  x = fmaf(sz.x, acc[i][nt][2 * h + c], zq);
                }
            }
        }
      } else {
        float acc[NT][4];
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const int mi = lane >> 3, row = (mi & 1) * 8 + (lane & 7), chunk = 2 * (ks & 3) + (mi >> 1);
          uint32_t a[4];
          ldmatrix_x4<false>(stage_addr + (ks >> 2) * 2048 + row * 128 + ((chunk ^ (row & 7)) << 4), a);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 bq = qf[(ks * NT + nt) * 32 + lane];
            mma_16816<BF16>(acc[nt], a[0], a[1], a[2], a[3], bq.x, bq.y, ks == 0);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[0][nt][c] = acc[nt][c] * p.scale_log2;
      }

      // ---- masks: the edges of the rows' windows, the end of the sequence or of the stream
      const bool cut = !(x0 + C::kTiles <= sinks_end || (x0 >= all_from && x0 + C::kTiles <= all_end));
      uint32_t dead = 0;
      if (cut) {
#pragma unroll
        for (int i = 0; i < C::kTiles; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = x0 + i < span.n_tiles ? span.tile_key(x0 + i) + row_a + 8 * h : 0x7fffffff;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int at = pos[nt][c];
                const bool see = key <= at && (key >= split_edge(p, at) || key < sinks);
                if (!see) s[i][nt][2 * h + c] = -INFINITY;
              }
            // a key that no row sees: its parameters may be anything
            if (!(key <= pos_max && (key >= low || key < sinks))) dead |= 1u << (2 * i + h);
          }
      }

      // ---- running maxima, lazy: a row's is brought up to date (and what was summed rescaled)
      // when an exponent lies more than 8 above it
      float mx[NT][2];
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = fmaxf(s[0][nt][c], s[0][nt][c + 2]);
#pragma unroll
          for (int i = 1; i < C::kTiles; ++i) x = fmax3(x, s[i][nt][c], s[i][nt][c + 2]);
          mx[nt][c] = x;
          grow |= fmaf(x, unit[nt][c], -m[nt][c]) > 8.f;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float top = group_max(mx[nt][c]) * unit[nt][c];
            const bool up = top > m[nt][c] + 8.f;
            const float alpha = up ? ex2_approx(m[nt][c] - top) : 1.f;
            m[nt][c] = up ? top : m[nt][c];
            l[nt][c] *= alpha;
#pragma unroll
            for (int gg = 0; gg < kGroups; ++gg) {
              csum[gg][nt][c] *= alpha;
              zsum[gg][nt][c] *= alpha;
            }
#pragma unroll
            for (int mt = 0; mt < kM; ++mt) {
              o[mt][nt][c] *= alpha;
              o[mt][nt][c + 2] *= alpha;
            }
          }
      }
      [[maybe_unused]] uint32_t par_v[C::kTiles][2][kGroups];
      if constexpr (Q4) {
#pragma unroll
        for (int i = 0; i < C::kTiles; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            params(i, h, 1, par_v[i][h]);
            if ((dead >> (2 * i + h)) & 1u)
#pragma unroll
              for (int gg = 0; gg < kGroups; ++gg) par_v[i][h][gg] = 0u;
          }
#pragma unroll
        for (int gg = 0; gg < kGroups; ++gg) {
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < C::kTiles; ++i)
            top = fmax3(top, unpack2<false>(par_v[i][0][gg]).x, unpack2<false>(par_v[i][1][gg]).x);
          if (__any_sync(0xffffffffu, top > big[gg])) {
            top = group_max(top);  // the same in all lanes
            const float r = __uint_as_float((__float_as_uint(top) & 0x7f800000u) + 0x00800000u);  // next power of two
            const float f = big[gg] / r;
            big[gg] = r;
            inv_big[gg] = 1.0f / r;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
              for (int c = 0; c < 2; ++c) csum[gg][nt][c] *= f;
#pragma unroll
              for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[gg * 4 + n][nt][c] *= f;
            }
          }
        }
      }

      // ---- P, its sums, and O^T += V^T P^T
#pragma unroll
      for (int i = 0; i < C::kTiles; ++i) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float pr = ex2_approx(fmaf(s[i][nt][c], unit[nt][c & 1], -m[nt][c & 1]));
            s[i][nt][c] = pr;
            l[nt][c & 1] += pr;
          }
        if constexpr (Q4) {
#pragma unroll
          for (int gg = 0; gg < kGroups; ++gg) {
            uint32_t bp[NT][2];
            [[maybe_unused]] uint32_t bq[NT][2];  // what P' was rounded by
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float2 sz = unpack2<false>(par_v[i][h][gg]);
              const float sv = sz.x * inv_big[gg];
              const float zv = fmaf(8.f, sz.x, sz.y);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const float w0 = s[i][nt][2 * h] * sv, w1 = s[i][nt][2 * h + 1] * sv;
                const uint32_t w = pack2<false>(w0, w1);
                if constexpr (!BF16) {
                  const float2 f = unpack2<false>(w);
                  bq[nt][h] = transpose_8x8(pack2<false>(w0 - f.x, w1 - f.y));
                }
                zsum[gg][nt][0] = fmaf(s[i][nt][2 * h], zv, zsum[gg][nt][0]);
                zsum[gg][nt][1] = fmaf(s[i][nt][2 * h + 1], zv, zsum[gg][nt][1]);
                bp[nt][h] = transpose_8x8(w);
              }
            }
            constexpr uint32_t kOnes = 0x3C003C00u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_16816<false>(csum[gg][nt], kOnes, kOnes, kOnes, kOnes, bp[nt][0], bp[nt][1]);
              if constexpr (!BF16) mma_16816<false>(csum[gg][nt], kOnes, kOnes, kOnes, kOnes, bq[nt][0], bq[nt][1]);
            }
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = *reinterpret_cast<const uint32_t*>(stage + i * C::kTileBytes + off_v[e] + gg * 32);
            // codes 0 .. 3 (w0, w2) and 4 .. 7 (w1, w3) of two keys each, key by key in a 16-bit half
            uint32_t w0 = __byte_perm(v[0], v[1], 0x5410), w1 = __byte_perm(v[0], v[1], 0x7632);
            uint32_t w2 = __byte_perm(v[2], v[3], 0x5410), w3 = __byte_perm(v[2], v[3], 0x7632);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const uint32_t mask = (n & 1) ? 0x00F000F0u : 0x000F000Fu;
              if (n == 2) {
                w0 >>= 8; w1 >>= 8; w2 >>= 8; w3 >>= 8;
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_16816<false>(o[gg * 4 + n][nt], w0 & mask, w1 & mask, w2 & mask, w3 & mask, bp[nt][0], bp[nt][1]);
                if constexpr (!BF16)
                  mma_16816<false>(o[gg * 4 + n][nt], w0 & mask, w1 & mask, w2 & mask, w3 & mask, bq[nt][0], bq[nt][1]);
              }
            }
          }
        } else {
          // bf16: P as the sum of two bf16 values (16 bits), a product each
          uint32_t bp[NT][2], bq[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t w = pack2<BF16>(s[i][nt][2 * h], s[i][nt][2 * h + 1]);
              bp[nt][h] = transpose_8x8(w);
              if constexpr (BF16) {
                const float2 f = unpack2<true>(w);
                bq[nt][h] = transpose_8x8(pack2<true>(s[i][nt][2 * h] - f.x, s[i][nt][2 * h + 1] - f.y));
              }
            }
#pragma unroll
          for (int mt = 0; mt < kM; ++mt) {
            const int mi = lane >> 3, row = (mi >> 1) * 8 + (lane & 7), chunk = 2 * (mt & 3) + (mi & 1);
            uint32_t a[4];
            ldmatrix_x4<true>(stage_addr + (kGroups + (mt >> 2)) * 2048 + row * 128 + ((chunk ^ (row & 7)) << 4), a);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_16816<BF16>(o[mt][nt], a[0], a[1], a[2], a[3], bp[nt][0], bp[nt][1]);
              if constexpr (BF16) mma_16816<BF16>(o[mt][nt], a[0], a[1], a[2], a[3], bq[nt][0], bq[nt][1]);
            }
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (k + C::kStages < mine) issue(k + C::kStages, st);
      if (++st == C::kStages) {
        st = 0;
        phase ^= 1u;
      }
    }
    // after an abort: let the copies in flight land
    for (int j = k; j < min(mine, k + C::kStages); ++j) {
      mbar_wait_drain_inline(bars + 8 * st, phase, p.timeout_ns);
      if (++st == C::kStages) {
        st = 0;
        phase ^= 1u;
      }
    }
    __syncthreads();  // every warp is done with the ring

    // ---- this warp's partial rows: o in units of 2^m, in natural channel order
    float* part = reinterpret_cast<float*>(smem) + warp * C::kRows * C::kPitch;
    float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = nt * 8 + 2 * t + c;
        float* row = part + r * C::kPitch;
        const float lsum = group_sum(l[nt][c]);
        if (g == 0) ml[warp * C::kRows + r] = make_float2(m[nt][c], lsum);
        if constexpr (Q4) {
#pragma unroll
          for (int gg = 0; gg < kGroups; ++gg) {
            const float base = fmaf(-8.f * big[gg], csum[gg][nt][c], group_sum(zsum[gg][nt][c]));
            const float f0 = big[gg] * 16777216.f, f1 = big[gg] * 1048576.f;  // even and odd codes
            float4 a, z;
            a.x = fmaf(f0, o[gg * 4 + 0][nt][c], base);
            a.y = fmaf(f1, o[gg * 4 + 1][nt][c], base);
            a.z = fmaf(f0, o[gg * 4 + 2][nt][c], base);
            a.w = fmaf(f1, o[gg * 4 + 3][nt][c], base);
            z.x = fmaf(f0, o[gg * 4 + 0][nt][c + 2], base);
            z.y = fmaf(f1, o[gg * 4 + 1][nt][c + 2], base);
            z.z = fmaf(f0, o[gg * 4 + 2][nt][c + 2], base);
            z.w = fmaf(f1, o[gg * 4 + 3][nt][c + 2], base);
            *reinterpret_cast<float4*>(row + gg * 64 + g * 8) = a;
            *reinterpret_cast<float4*>(row + gg * 64 + g * 8 + 4) = z;
          }
        } else {
#pragma unroll
          for (int mt = 0; mt < kM; ++mt) {
            row[mt * 16 + g] = o[mt][nt][c];
            row[mt * 16 + g + 8] = o[mt][nt][c + 2];
          }
        }
      }
    __syncthreads();

    // ---- sum over the warps: the item's rows, or this part of them
    const bool whole = ca == 0 && cb == n_chunks;
    const float* rows_of = reinterpret_cast<const float*>(smem);
    float* dst = p.part + (2LL * blockIdx.x + (ca == 0 ? 1 : 0)) * (C::kRows * C::kPitch);  // of a part
    for (int e = threadIdx.x; e < rows * (D / 4); e += 256) {
      const int r = e / (D / 4), c4 = e % (D / 4) * 4;
      const SplitSum a = split_sum_fixed<C::kWarps>(
          [&](int w) { return ml[w * C::kRows + r]; },
          [&](int w) { return *reinterpret_cast<const float4*>(rows_of + (w * C::kRows + r) * C::kPitch + c4); });
      if (whole) {
        split_store<D, BF16>(p, b, hk, chunk_row0 + r, c4, a);
      } else {
        *reinterpret_cast<float4*>(dst + r * C::kPitch + c4) = a.o;
        if (c4 == 0) *reinterpret_cast<float2*>(dst + r * C::kPitch + D) = make_float2(a.m, a.l);
      }
    }
    if (p.part == nullptr) break;
    if (!whole) {
      // n CTAs from c1 on hold parts of the item: c1 its first, in its second slot
      int c1, n;
      if (parts > 0) {
        c1 = blockIdx.x - blockIdx.x % parts;
        const int length = (n_chunks + parts - 1) / parts;
        n = (n_chunks + length - 1) / length;
      } else {
        const long long x0 = run - ca;
        c1 = (int)(x0 / run_length);
        n = (int)((x0 + n_chunks - 1) / run_length) - c1 + 1;
      }
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) *last_part = split_arrive(p.arrived + c1, p.nonce, n);
      __syncthreads();
      if (*last_part) {
        __threadfence();
        for (int e = threadIdx.x; e < rows * (D / 4); e += 256) {
          const int r = e / (D / 4), c4 = e % (D / 4) * 4;
          auto row = [&](int i) -> const float* {
            return p.part + ((2LL * (c1 + i) + (i == 0 ? 1 : 0)) * C::kRows + r) * C::kPitch;
          };
          split_store<D, BF16>(p, b, hk, chunk_row0 + r, c4, split_sum(
              n, [&](int i) { return __ldcg(reinterpret_cast<const float2*>(row(i) + D)); },
              [&](int i) { return __ldcg(reinterpret_cast<const float4*>(row(i) + c4)); }));
        }
      }
    }
    if (parts > 0) break;
    run += cb - ca;
    fence_proxy_async_smem();  // the partials' shared memory becomes the ring again
    __syncthreads();
    if (run >= run_end) break;
    if (run >= place.begin + (long long)n_chunks * p.Hkv * p.row_chunks) {  // the next request that has keys
      place.begin = run;
      do ++place.b;
      while (place.b < p.B - 1 && split_span<Q4>(p, place.b).n_tiles == 0);
    }
  }
}

}  // namespace attn_b200
