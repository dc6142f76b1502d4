// q4_cache.cuh -- the paged key/value cache held in 4 bits: its layout, the kernel that
// quantises new tokens into it and the kernel that reads it back (sm_100a).
//
// A group is 64 consecutive channels of one token's K (or V) in one head.  With lo and hi
// its smallest and largest element,
//   zero = fp16(lo),  scale = fp16((hi - lo) / 15),
//   code = clamp(round_to_even((x - zero) / scale), 0, 15)   (0 where scale = 0),
// and the code stands for zero + scale * code.  Groups of one token and head need no
// statistics of other tokens, so a token is quantised once, as it is written.  4.5 bits an
// element with the parameters.
//
// Layout: uint8 [num_blocks, Hkv, page_size, 9 d / 8].  The bytes of one head's page are a
// run of tiles of T = min(page_size, 16) tokens, each
//   K codes [T][d/2] | V codes [T][d/2] | params [T][K, V][d/64][scale, zero] fp16,
// channel 2i of a row in the low half of byte i, 2i + 1 in the high half.  A tile is what
// the attention kernel fetches in one bulk copy (2304 bytes at d = 128), and its 16 tokens
// are one MMA's rows.
#pragma once

#include "sm100_ptx.cuh"

namespace attn_b200 {

constexpr int kQ4Group = 64;    // channels that share a scale and a zero
constexpr int kQ4MaxTile = 16;  // tokens of a tile (8 in 8-token pages)

template <int D>
struct Q4Layout {
  static constexpr int kGroups = D / kQ4Group;
  static constexpr int kRowBytes = D / 2;            // a token's K (or V) codes
  static constexpr int kParBytes = 2 * kGroups * 4;  // a token's parameters, K then V
  static constexpr int kTokenBytes = 2 * kRowBytes + kParBytes;
  static_assert(kTokenBytes == 9 * D / 8, "4.5 bits an element");
};

// Where the cache row of logical position `pos` of a request lies: the tile's first byte and
// the token's place in it.  `block` is the page that the request's table row names.
struct Q4Place {
  long long tile;  // byte offset of the tile
  int row;         // token within the tile
};

template <int D>
__device__ __forceinline__ Q4Place q4_place(int block, int head, int in_page, int Hkv, int page_size) {
  const int T = min(page_size, kQ4MaxTile);
  const int tile = in_page / T;
  Q4Place p;
  p.tile = (((long long)block * Hkv + head) * page_size + (long long)tile * T) * Q4Layout<D>::kTokenBytes;
  p.row = in_page - tile * T;
  return p;
}

struct Q4WriteParams {
  const void* k;           // [B, Ln, Hkv, d]
  const void* v;           // [B, Ln, Hkv, d]
  uint8_t* cache;
  const int* block_table;  // [B, max_blocks]
  const int* seq_lens;     // [B], new tokens included
  const int* new_lens;     // [B] or nullptr (Ln each)
  int* status;
  int B, Ln, Hkv, num_blocks, page_size, max_blocks;
};

// Code of x (finite) in a group: nearest even in the exact quotient.  2 x against
// 2 zero + (2 c + 1) scale in double: x alone is exact whatever its exponent, and the right side,
// made of fp16 values, is a multiple of 2^-24 below 2^19, so a tie is seen as one and nothing else is.
// (x - zero would not be exact: a bf16 x of 2^-60 vanishes beside a zero of -1.)
__device__ __forceinline__ int q4_code_exact(float x, float zero, float scale, float t) {
  const double x2 = 2.0 * (double)x, zero2 = 2.0 * (double)zero;
  int c = (int)floorf(fminf(fmaxf(t, -1.f), 16.f) + 0.5f) - 1;  // one or two below the answer
  c = max(c, -2);
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {  // at most three borders lie between c and the answer
    const double border = fma((double)(2 * c + 1), (double)scale, zero2);
    if (x2 > border || (x2 == border && (c & 1))) ++c;
    else break;
  }
  return min(max(c, 0), 15);
}

// A warp quantises a token: a lane takes 16 channels of a head's K or V at a time (K of all
// heads, then V), the four lanes of a group share its smallest and largest element by shuffles.
// Reads run along the token's heads, contiguously; a lane stores 8 bytes of codes.  A token is
// placed once per warp, so the lanes do no divisions.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) q4_write_kernel(const Q4WriteParams p) {
  using L = Q4Layout<D>;
  constexpr int kParts = D / 16;
  const int lane = threadIdx.x & 31, i = blockIdx.x * 8 + (threadIdx.x >> 5), b = blockIdx.y;
  if (i >= p.Ln) return;
  const long long most = (long long)p.max_blocks * p.page_size;
  const int n = p.new_lens ? min(max(p.new_lens[b], 0), p.Ln) : p.Ln;
  // a length past the table is not cut off here: its last tokens would land on earlier tokens' rows
  const long long pos = (long long)max(p.seq_lens[b], 0) - n + i;
  if (i >= n || pos < 0 || pos >= most) return;
  const int page = (int)(pos / p.page_size), in_page = (int)(pos - (long long)page * p.page_size);
  const int block = p.block_table[(long long)b * p.max_blocks + page];
  if (block < 0 || block >= p.num_blocks) return;  // never writes outside the cache, or another page
  const int T = min(p.page_size, kQ4MaxTile);
  const int pieces = p.Hkv * kParts;
  const long long token = ((long long)b * p.Ln + i) * p.Hkv * D;
  auto source = [&](int e) -> const uint32_t* {  // 16 elements
    return reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(e >= pieces ? p.v : p.k) + token +
                                             (e >= pieces ? e - pieces : e) * 16);
  };
  uint4 a = make_uint4(0u, 0u, 0u, 0u), c = a;
  if (lane < 2 * pieces) {
    a = __ldg(reinterpret_cast<const uint4*>(source(lane)));
    c = __ldg(reinterpret_cast<const uint4*>(source(lane)) + 1);
  }
  for (int e = lane; e < 2 * pieces; e += 32) {  // a multiple of 4: groups of four lanes stay together
    const int left = 2 * pieces - (e - lane);
    const unsigned live = left >= 32 ? 0xffffffffu : (1u << left) - 1u;
    const bool is_v = e >= pieces;
    const int piece = is_v ? e - pieces : e, head = piece / kParts, part = piece % kParts;
    const uint32_t* src32 = source(e);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
    if (e + 32 < 2 * pieces) {  // the next piece's elements, while this one is worked on
      const uint4* next = reinterpret_cast<const uint4*>(source(e + 32));
      a = __ldg(next);
      c = __ldg(next + 1);
    }
    // magnitudes with no finite fp16 value, of two elements at a time
    uint32_t mag = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) mag = __vmaxu2(mag, w[e] & 0x7FFF7FFFu);
    const bool bad = max(mag & 0xFFFFu, mag >> 16) >= (BF16 ? kBf16NoF16 : 0x7C00u);
    float x[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 f = unpack2<BF16>(w[e]);
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
    if (bad) {  // NaN becomes -65504: the cache stays finite
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = fminf(fmaxf(x[e], -65504.f), 65504.f);
    }
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      lo = -fmax3(-lo, -x[e], -x[e + 1]);
      hi = fmax3(hi, x[e], x[e + 1]);
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(live, lo, off));
      hi = fmaxf(hi, __shfl_xor_sync(live, hi, off));
    }
    const __half zero_h = __float2half_rn(lo);
    // (hi - lo) / 15 correctly rounded in double (a reciprocal product and one residual step),
    // then to fp16: a quotient that is exactly between two fp16 values stays exactly there
    const double span = (double)hi - (double)lo;
    double quo = span * (1.0 / 15.0);
    quo = fma(fma(-15.0, quo, span), 1.0 / 15.0, quo);
    const __half scale_h = __double2half(quo);
    const float zero = __half2float(zero_h), scale = __half2float(scale_h);
    const float inv = scale > 0.f ? 1.0f / scale : 0.f;

    // Rounding by 1.5 * 2^23, in whose sum the code is the low mantissa bits: a conversion to
    // integer takes the slow pipe.  Eight codes of a word are added up as t_i 16^i, the constant's
    // share taken off at the end (all mod 2^32).
    constexpr float kRound = 12582912.f;
    constexpr uint32_t kRoundBits = 0x4B400000u * 0x11111111u;
    float far = 0.f;  // largest distance of a quotient (within the codes) from its code
    uint32_t code[2] = {0u, 0u};
#pragma unroll
    for (int e = 15; e >= 0; --e) {
      const float q = fminf(fmaxf((x[e] - zero) * inv, 0.f), 15.f);
      const float t = q + kRound;
      far = fmaxf(far, fabsf(q - (t - kRound)));
      code[e >> 3] = code[e >> 3] * 16u + __float_as_uint(t);
    }
    uint2 out = make_uint2(code[0] - kRoundBits, code[1] - kRoundBits);
    // The quotient above is off by at most |q| * 3 * 2^-24 < 3e-6 (three roundings, q <= 15.01),
    // so where it lies farther than that from a border between two codes its rounding is the
    // exact quotient's.  Ties are 8 elements in 10000 of bf16 rows, so a warp of four meets one.
    if (scale > 0.f && far > 0.5f - 4e-6f) {
      uint32_t near = 0;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float q = fminf(fmaxf((x[e] - zero) * inv, 0.f), 15.f);
        if (fabsf(q - ((q + kRound) - kRound)) > 0.5f - 4e-6f) near |= 1u << e;
      }
      for (; near != 0; near &= near - 1) {
        const int e = __ffs(near) - 1;
        const float2 f = unpack2<BF16>(src32[e >> 1]);
        const float y = fminf(fmaxf((e & 1) ? f.y : f.x, -65504.f), 65504.f);
        const uint32_t c = (uint32_t)q4_code_exact(y, zero, scale, (y - zero) * inv);
        uint32_t& word = e < 8 ? out.x : out.y;
        word = (word & ~(15u << (4 * (e & 7)))) | c << (4 * (e & 7));
      }
    }
    const Q4Place at = q4_place<D>(block, head, in_page, p.Hkv, p.page_size);
    uint8_t* tile = p.cache + at.tile;
    *reinterpret_cast<uint2*>(tile + ((is_v ? T : 0) + at.row) * L::kRowBytes + part * 8) = out;
    if (part % 4 == 0) {
      const __half2 par = __halves2half2(scale_h, zero_h);
      *reinterpret_cast<__half2*>(tile + 2 * T * L::kRowBytes + at.row * L::kParBytes +
                                  ((is_v ? L::kGroups : 0) + part / 4) * 4) = par;
    }
    if (bad) atomicCAS(p.status, 0, kStatusRange);
  }
}

struct Q4ReadParams {
  const uint8_t* cache;
  const int* block_table;
  const int* seq_lens;
  void* k;  // [B, Nmax, Hkv, d]
  void* v;
  int B, Nmax, Hkv, num_blocks, page_size, max_blocks;
};

// A warp reads kQ4ReadRows rows of a request back: a lane writes 8 channels (16 bytes) of a head's
// K and V at a time, the values that the codes stand for, rounded once to the output type, so a
// warp's stores are whole lines (16 channels a lane, in two stores 32 bytes apart, took 40 us
// where this takes 30: 8000 rows of 8 heads, 4 requests); rows at or past the request's length
// are zero.  The rows are placed once per warp, and their loads are issued together.
constexpr int kQ4ReadRows = 4;

template <int D, bool BF16>
__global__ void __launch_bounds__(256) q4_read_kernel(const Q4ReadParams p) {
  using L = Q4Layout<D>;
  constexpr int kParts = D / 8, R = kQ4ReadRows;
  const int lane = threadIdx.x & 31, i0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * R, b = blockIdx.y;
  if (i0 >= p.Nmax) return;
  const int len = (int)min((long long)p.seq_lens[b], (long long)p.max_blocks * p.page_size);
  const int T = min(p.page_size, kQ4MaxTile), rows = min(R, p.Nmax - i0);
  const int page = i0 / p.page_size;
  const int block = i0 < len ? min(max(p.block_table[(long long)b * p.max_blocks + page], 0), p.num_blocks - 1) : 0;
  // kQ4ReadRows divides the tokens of a tile, so the rows lie in one
  const Q4Place at = q4_place<D>(block, 0, i0 - page * p.page_size, p.Hkv, p.page_size);
  const uint8_t* tile = p.cache + at.tile;
  const long long head_bytes = (long long)p.page_size * L::kTokenBytes;
  const int pieces = p.Hkv * kParts;
  for (int piece = lane; piece < pieces; piece += 32) {
    const uint8_t* src = tile + piece / kParts * head_bytes;
    const int part = piece % kParts;
    uint32_t code[2][R], par[2][R];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        code[y][r] = par[y][r] = 0u;
        if (i0 + r < len) {
          const int row = at.row + r;
          code[y][r] = __ldg(reinterpret_cast<const uint32_t*>(src + (y * T + row) * L::kRowBytes + part * 4));
          par[y][r] = __ldg(reinterpret_cast<const uint32_t*>(src + 2 * T * L::kRowBytes + row * L::kParBytes +
                                                              (y * L::kGroups + part / 8) * 4));
        }
      }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= rows) break;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float2 sz = unpack2<false>(par[y][r]);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t word = code[y][r] >> (8 * e);
          // scale * code is exact in fp32 (15 bits); one rounding in the sum, one to the output type
          w[e] = pack2<BF16>(fmaf(sz.x, (float)(word & 15u), sz.y), fmaf(sz.x, (float)((word >> 4) & 15u), sz.y));
        }
        reinterpret_cast<uint4*>(y ? p.v : p.k)[((long long)b * p.Nmax + i0 + r) * pieces + piece] =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

}  // namespace attn_b200
