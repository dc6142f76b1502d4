// attn_window.cu -- entry points of attention over a sliding window with sink tokens and of
// the 4-bit paged cache (declared in include/attn.h): argument checks and launches.
#include <unistd.h>

#include <algorithm>
#include <atomic>
#include <chrono>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "sm100_ptx_window.cuh"

#include "attn_host.h"
#include "q4_cache.cuh"
#include "split_sm100.cuh"
#include "window_bwd_sm100.cuh"
#include "window_fwd_sm100.cuh"

using namespace attn_b200;

namespace {

// Grouped heads, sizes, dtype, scale and alignment shared by the window entry points.
int check_window(const void* q, const void* k, const void* v, int B, int H, int Hkv, int Nq, int Nk, int d,
                 int window, int sinks, float scale, int dtype) {
  if (!q || !k || !v) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || H <= 0 || Hkv <= 0 || Nq <= 0 || Nk <= 0 || d <= 0) return ATTN_ERR_INVALID_ARG;
  if (H % Hkv != 0 || window <= 0 || sinks < 0 || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_UNSUPPORTED;
  if (host_misaligned(q, 16) || host_misaligned(k, 16) || host_misaligned(v, 16)) return ATTN_ERR_INVALID_ARG;
  // tensor-map limit: the batch stride stays below 2^40 bytes
  const unsigned long long row = 2ull * d;
  if (row * Nq * H >= (1ull << 40) || row * Nk * Hkv >= (1ull << 40)) return ATTN_ERR_INVALID_ARG;
  // rows of any kind are counted in 32 bits
  if ((long long)B * Nq * H >= (1LL << 31) || (long long)B * Nk * Hkv >= (1LL << 31)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

bool page_ok(int page_size) {
  return page_size < 128 ? (page_size >= 8 && 128 % page_size == 0) : (page_size % 128 == 0);
}

// The cache of the q4 entry points: sizes, layout limits and alignment.
int check_q4(const void* cache, const int* block_table, const int* seq_lens, int B, int Hkv, int d, int num_blocks,
             int page_size, int max_blocks) {
  if (!cache || !block_table || !seq_lens) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hkv <= 0 || d <= 0 || num_blocks <= 0 || page_size <= 0 || max_blocks <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (!page_ok(page_size)) return ATTN_ERR_UNSUPPORTED;
  if ((long long)num_blocks * page_size >= (1LL << 31) || (long long)max_blocks * page_size >= (1LL << 31))
    return ATTN_ERR_INVALID_ARG;
  if (host_misaligned(cache, 16) || host_misaligned(block_table, 4) || host_misaligned(seq_lens, 4))
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

size_t q4_bytes(int Hkv, int d, int num_blocks, int page_size) {
  return (size_t)num_blocks * page_size * Hkv * (9 * d / 8);
}

bool dtype_ok(int dtype) { return dtype == ATTN_F16 || dtype == ATTN_BF16; }

int launched() { return cudaGetLastError() == cudaSuccess ? ATTN_OK : cuda_failed(); }

constexpr int kMaxGridY = 65535;  // requests of a cache call

// Items of at most this many keys take a CTA each and no workspace.  One token, 128 channels, dense
// bf16 | 4-bit, parts or runs against a CTA an item (us, inputs not in L2): 4 items of 512 keys 12.9 / 10.2 |
// 12.9 / 12.3, of 2048 17.0 / 18.4 | 17.0 / 20.5; 128 items of 512 17.0 / 14.3 | 17.0 / 12.3; 512 items of
// 512 45.7 / 41.0 | 39.5 / 28.7.  Equal items of 1024 keys would still gain (4 items 14.9 / 12.3); the keys
// counted here are the most that an item can have, and past some hundred a CTA with one of them would
// work on while those of the short ones have ended.
constexpr long long kDirectKeys = 512;

// Calls f(head_dim, is bf16) with both as compile-time constants.
template <typename F>
int by_type(int d, int dtype, F&& f) {
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (dtype == ATTN_BF16) return d == 128 ? f(D128{}, std::true_type{}) : f(D64{}, std::true_type{});
  return d == 128 ? f(D128{}, std::false_type{}) : f(D64{}, std::false_type{});
}

// Largest power of two that divides the heads of a group, at most 16: the heads that share a
// Q tile (a tile of 128 rows then spans 128 / pack positions).
int pack_log2(int group) {
  int lg = 0;
  while (lg < 4 && group % (2 << lg) == 0) ++lg;
  return lg;
}

template <int D, bool BF16>
int launch_window_fwd(const DeviceInfo& dev, const void* q, const void* k, const void* v, void* out, float* lse, int B,
                      int H, int Hkv, int Nq, int Nk, int window, int sinks, float scale, cudaStream_t stream) {
  using C = WindowFwdCfg<D>;
  WindowFwdParams p;
  const int dtype = BF16 ? ATTN_BF16 : ATTN_F16;
  p.group = H / Hkv;
  p.lg_pack = pack_log2(p.group);
  const int pack = 1 << p.lg_pack, rows = 128 >> p.lg_pack;
  if (int rc = host_encode_bnhd(&p.tm_q, q, B, Nq, H, D, dtype, rows, pack)) return rc;
  if (int rc = host_encode_bnhd(&p.tm_k, k, B, Nk, Hkv, D, dtype, 128)) return rc;
  if (int rc = host_encode_bnhd(&p.tm_v, v, B, Nk, Hkv, D, dtype, 128)) return rc;
  if (int rc = host_encode_bnhd(&p.tm_k8, k, B, Nk, Hkv, D, dtype, 8)) return rc;
  if (int rc = host_encode_bnhd(&p.tm_v8, v, B, Nk, Hkv, D, dtype, 8)) return rc;
  if (int rc = host_encode_bnhd(&p.tm_o, out, B, Nq, H, D, dtype, rows, pack)) return rc;
  p.out = out;
  p.lse = lse;
  p.status = dev.status_ptr;
  p.B = B;
  p.H = H;
  p.Nq = Nq;
  p.Nk = Nk;
  p.window = window;
  p.sinks = sinks;
  p.n_pairs = (Nq + 2 * rows - 1) / (2 * rows);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.timeout_ns = host_timeout_ns();
  p.inject = host_inject();
  const long long pairs = (long long)B * (H / pack) * p.n_pairs;
  // Units are of one size, so they end in a partial wave; when it would fill at most half of
  // the SMs (or there is no full one), its pairs run as units of one tile in about half the time.
  const long long rem = pairs % dev.sm_count;
  p.n_split = 2 * rem <= dev.sm_count ? (int)rem : 0;
  const long long units = pairs + p.n_split;
  if (units >= (1LL << 31)) return ATTN_ERR_INVALID_ARG;
  if (p.n_split > 0) {  // the kernel without one-tile units keeps its registers for the pairs
    if (int rc = host_raise_smem<attn_window_fwd_kernel<D, BF16, true>>(dev, C::kSmemBytes)) return rc;
    attn_window_fwd_kernel<D, BF16, true><<<(unsigned)units, C::kThreads, C::kSmemBytes, stream>>>(p);
  } else {
    if (int rc = host_raise_smem<attn_window_fwd_kernel<D, BF16, false>>(dev, C::kSmemBytes)) return rc;
    attn_window_fwd_kernel<D, BF16, false><<<(unsigned)units, C::kThreads, C::kSmemBytes, stream>>>(p);
  }
  return launched();
}

// 48 bits that no other launch is likely to have, the low 16 being 0: a mixed counter from a
// start that differs from process to process (the mixing is the finaliser of the splitmix64
// generator).
unsigned long long launch_nonce() {
  static std::atomic<unsigned long long> next{
      (unsigned long long)std::chrono::high_resolution_clock::now().time_since_epoch().count() ^
      ((unsigned long long)getpid() << 40)};
  unsigned long long x = next.fetch_add(0x9E3779B97F4A7C15ull);
  x = (x ^ (x >> 30)) * 0xBF58476D1CE4E5B9ull;
  x = (x ^ (x >> 27)) * 0x94D049BB133111EBull;
  return (x ^ (x >> 31)) << 16;
}

// Workspace, stream-ordered.  It comes from a pool of the library's own that keeps up to
// kPoolKeep bytes between calls: the default pool gives everything back to the system at each
// synchronisation, after which a call waited 0.1 to 8 ms on the host for its few megabytes.
// Under capture the graph owns the memory.
constexpr unsigned long long kPoolKeep = 256ull << 20;

int take_workspace(const DeviceInfo& dev, void** ptr, size_t bytes, cudaStream_t stream) {
  static std::mutex mutex;
  static cudaMemPool_t pools[kHostMaxDevices] = {};
  cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &capturing) != cudaSuccess) return cuda_failed();
  if (capturing != cudaStreamCaptureStatusNone)
    return cudaMallocAsync(ptr, bytes, stream) == cudaSuccess ? ATTN_OK : cuda_failed();
  cudaMemPool_t pool = nullptr;
  {
    std::lock_guard<std::mutex> lock(mutex);
    if (pools[dev.device] == nullptr) {
      cudaMemPoolProps props{};
      props.allocType = cudaMemAllocationTypePinned;
      props.location.type = cudaMemLocationTypeDevice;
      props.location.id = dev.device;
      cudaMemPool_t made = nullptr;
      if (cudaMemPoolCreate(&made, &props) != cudaSuccess) return cuda_failed();
      cuuint64_t keep = kPoolKeep;
      if (cudaMemPoolSetAttribute(made, cudaMemPoolAttrReleaseThreshold, &keep) != cudaSuccess) {
        cudaMemPoolDestroy(made);
        return cuda_failed();
      }
      pools[dev.device] = made;
    }
    pool = pools[dev.device];
  }
  return cudaMallocFromPoolAsync(ptr, bytes, pool, stream) == cudaSuccess ? ATTN_OK : cuda_failed();
}

// One launch of the split-over-keys kernel; p holds what does not follow from the sizes.
template <int D, bool BF16, bool Q4, int NT>
int launch_split(const DeviceInfo& dev, SplitParams& p, cudaStream_t stream) {
  using C = SplitCfg<D, Q4, NT>;
  if (int rc = host_raise_smem<attn_split_kernel<D, BF16, Q4, NT>>(dev, C::kSmemBytes)) return rc;
  const long long rows = (long long)p.Lq * (p.H / p.Hkv);
  p.row_chunks = (int)((rows + C::kRows - 1) / C::kRows);
  const long long items = (long long)p.B * p.Hkv * p.row_chunks;
  if (items >= (1LL << 31)) return ATTN_ERR_INVALID_ARG;
  // keys that an item can have to read
  long long keys = p.Nk;
  if (p.window > 0) keys = std::min<long long>(keys, (long long)p.window + p.Lq + std::min(p.sinks, p.Nk));
  const int slots = dev.sm_count * C::kCtas;
  if (keys <= kDirectKeys) {
    attn_split_kernel<D, BF16, Q4, NT><<<(unsigned)items, 256, C::kSmemBytes, stream>>>(p);
    return launched();
  }
  const size_t part_bytes = 2ull * slots * C::kPartBytes;  // a multiple of 8
  void* ws = nullptr;
  if (int rc = take_workspace(dev, &ws, part_bytes + 8ull * slots, stream)) return rc;
  p.part = static_cast<float*>(ws);
  p.arrived = reinterpret_cast<unsigned long long*>(static_cast<uint8_t*>(ws) + part_bytes);
  p.nonce = launch_nonce();
  attn_split_kernel<D, BF16, Q4, NT><<<slots, 256, C::kSmemBytes, stream>>>(p);
  int rc = launched();
  if (cudaFreeAsync(ws, stream) != cudaSuccess) rc = cuda_failed();
  return rc;
}

// Query rows of a key/value head up to which attn_fwd_window splits the keys over the CTAs; past
// it the tiles' kernel runs.  At 128 channels, 32 query heads over 8, 32 rows split against 36
// rows tiled, which take no longer than 32 would (us, inputs not in L2): 2 requests, 4096 of 8192
// keys 37.4 / 71.7; 16 requests, 1024 of 4096 keys 32.5 / 30.0; 64 requests, 2048 keys 144.0 /
// 153.6.  64 rows would be two items that each read the keys: about twice the tiles' time in the second.
constexpr long long kSplitRows = 32;

// 8, 16 or 32 query rows an item: the fewest that hold the rows of a key/value head.
template <int D, bool BF16, bool Q4>
int launch_split_rows(const DeviceInfo& dev, SplitParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.Lq * (p.H / p.Hkv);
  if (rows <= 8) return launch_split<D, BF16, Q4, 1>(dev, p, stream);
  if (rows > 16) return launch_split<D, BF16, Q4, 4>(dev, p, stream);
  return launch_split<D, BF16, Q4, 2>(dev, p, stream);
}

// Steps of a unit of the keys' launch below which it is not split further.  With 1, 2, 4, 8, 16 (us,
// inputs not in L2, 2 heads of keys and groups of 4): 1000 tokens, window 256, 64 channels fp16 51.8 45.7
// 39.5 45.6 58.0, 128 channels bf16 74.3 60.0 45.7 51.8 66.1; 700 tokens, every key, one head 43.6 35.4 37.5
// 43.6 49.8; 2 x 512 tokens, 4 heads, window 128 78.4 66.1 60.0 57.9 58.0.  From 2000 tokens of 8 heads on
// the share of an SM decides (150 to 156 with any).
constexpr long long kBwdMinSteps = 4;

template <int D, bool BF16>
int launch_window_bwd(const DeviceInfo& dev, const void* q, const void* k, const void* v, const void* o,
                      const long long (&o_strides)[3], const void* dout, const float* lse, void* dq, void* dk, void* dv, int B, int H, int Hkv, int Nq,
                      int Nk, int window, int sinks, float scale, cudaStream_t stream) {
  using C = WindowBwdCfg<D>;
  if (int rc = host_raise_smem<attn_window_bwd_kernel<D, BF16, false>>(dev, C::kSmemBytes)) return rc;
  if (int rc = host_raise_smem<attn_window_bwd_kernel<D, BF16, true>>(dev, C::kSmemBytes)) return rc;
  const int dtype = BF16 ? ATTN_BF16 : ATTN_F16, group = H / Hkv;
  WindowBwdParams pq{}, pk{};
  pq.lg_pack = pack_log2(group);
  const int pack = 1 << pq.lg_pack, rows = 128 >> pq.lg_pack;
  if (int rc = host_encode_bnhd(&pq.tm_x1, q, B, Nq, H, D, dtype, rows, pack)) return rc;
  if (int rc = host_encode_bnhd(&pq.tm_x2, dout, B, Nq, H, D, dtype, rows, pack)) return rc;
  if (int rc = host_encode_bnhd(&pq.tm_y1, k, B, Nk, Hkv, D, dtype, 128)) return rc;
  if (int rc = host_encode_bnhd(&pq.tm_y2, v, B, Nk, Hkv, D, dtype, 128)) return rc;
  if (int rc = host_encode_bnhd(&pq.tm_y1_8, k, B, Nk, Hkv, D, dtype, 8)) return rc;
  if (int rc = host_encode_bnhd(&pq.tm_y2_8, v, B, Nk, Hkv, D, dtype, 8)) return rc;
  if (int rc = host_encode_bnhd(&pk.tm_x1, k, B, Nk, Hkv, D, dtype, 128)) return rc;
  if (int rc = host_encode_bnhd(&pk.tm_x2, v, B, Nk, Hkv, D, dtype, 128)) return rc;
  if (int rc = host_encode_bnhd(&pk.tm_y1, q, B, Nq, H, D, dtype, 128)) return rc;
  if (int rc = host_encode_bnhd(&pk.tm_y2, dout, B, Nq, H, D, dtype, 128)) return rc;
  pq.lse = lse;
  pq.status = dev.status_ptr;
  pq.B = B; pq.H = H; pq.Hkv = Hkv; pq.Nq = Nq; pq.Nk = Nk;
  pq.window = window;
  pq.sinks = sinks;
  pq.scale = scale;
  pq.scale_log2 = scale * 1.4426950408889634f;
  pq.timeout_ns = host_timeout_ns();
  pq.inject = pk.inject = host_inject();
  pk.lse = pq.lse; pk.status = pq.status;
  pk.B = B; pk.H = H; pk.Hkv = Hkv; pk.Nq = Nq; pk.Nk = Nk;
  pk.window = window; pk.sinks = sinks; pk.scale = scale; pk.scale_log2 = pq.scale_log2; pk.timeout_ns = pq.timeout_ns;
  pq.o = o;
  pq.o_batch = o_strides[0];
  pq.o_query = o_strides[1];
  pq.o_head = o_strides[2];
  pq.g1 = dq;
  pk.g1 = dv;
  pk.g2 = dk;
  pq.n_xtiles = (Nq + rows - 1) / rows;
  pk.n_xtiles = (Nk + 127) / 128;
  const long long q_units = (long long)B * (H / pack) * pq.n_xtiles;

  // Units of the keys' launch of at most half an SM's share of the steps (a tile with sinks is
  // seen by every later query: many times the others' steps), if more than kBwdMinSteps.
  const long long heads = (long long)B * Hkv;
  pk.sink_tiles = (int)(((long long)std::min(sinks, Nk) + 127) / 128);
  const long long rest_tiles = pk.n_xtiles - pk.sink_tiles;
  const long long sink_steps = (long long)group * ((Nq + 127) / 128);
  const long long steps = (long long)group * ((std::min<long long>(Nq, (long long)window + 127) + 127) / 128);
  const long long total = heads * (pk.sink_tiles * sink_steps + rest_tiles * steps);
  const long long most = std::max(kBwdMinSteps, total / (2LL * dev.sm_count));
  pk.sink_splits = (int)((sink_steps + most - 1) / most);
  pk.splits = (int)((steps + most - 1) / most);
  const long long sink_units = heads * pk.sink_tiles * pk.sink_splits, rest_units = heads * rest_tiles * pk.splits;
  const long long parts = (pk.sink_splits > 1 ? sink_units : 0) + (pk.splits > 1 ? rest_units : 0);
  const long long joined = (pk.sink_splits > 1 ? heads * pk.sink_tiles : 0) + (pk.splits > 1 ? heads * rest_tiles : 0);
  constexpr int kJoinBlocks = 128 * (D / 4) / 256;  // of a tile
  if (q_units >= (1LL << 31) || sink_units + rest_units >= (1LL << 31) || joined * kJoinBlocks >= (1LL << 31))
    return ATTN_ERR_INVALID_ARG;

  const int n_kblocks = (Nk + 127) / 128;
  const long long bound_blocks = heads * n_kblocks, n_qmax = 2 * heads * ((Nq + 127) / 128);
  if (bound_blocks >= (1LL << 31)) return ATTN_ERR_INVALID_ARG;
  const size_t dsum_bytes = ((size_t)B * H * Nq * 4 + 255) / 256 * 256, part_bytes = (size_t)parts * 256 * D * 4;
  const size_t vmax_bytes = BF16 ? 0 : ((size_t)bound_blocks * 4 + 255) / 256 * 256;
  void* ws = nullptr;
  if (int rc = take_workspace(dev, &ws, dsum_bytes + part_bytes + vmax_bytes + (BF16 ? 0 : n_qmax * 4), stream)) return rc;
  uint8_t* at = static_cast<uint8_t*>(ws);
  pq.dsum = pk.dsum = reinterpret_cast<float*>(at);
  pk.part = reinterpret_cast<float*>(at + dsum_bytes);
  pq.vmax = pk.vmax = reinterpret_cast<float*>(at + dsum_bytes + part_bytes);
  pq.qmax = pk.qmax = reinterpret_cast<unsigned*>(at + dsum_bytes + part_bytes + vmax_bytes);
  int rc = ATTN_OK;
  if constexpr (!BF16) {
    attn_window_bwd_kernel_bounds<D><<<(unsigned)bound_blocks, 256, 0, stream>>>(
        v, reinterpret_cast<float*>(at + dsum_bytes + part_bytes), pq.qmax, Hkv, Nk, n_kblocks, n_qmax);
    rc = launched();
  }
  // The later launches may start while the one before ends (programmatic dependent launch); they
  // wait for its end before they read what it wrote.
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = BF16 ? 0 : 1;
  if (rc == ATTN_OK) {
    cfg.gridDim = dim3((unsigned)q_units);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    if (cudaLaunchKernelEx(&cfg, attn_window_bwd_kernel<D, BF16, false>, pq) != cudaSuccess) rc = cuda_failed();
  }
  cfg.numAttrs = 1;
  if (rc == ATTN_OK) {
    cfg.gridDim = dim3((unsigned)(sink_units + rest_units));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    if (cudaLaunchKernelEx(&cfg, attn_window_bwd_kernel<D, BF16, true>, pk) != cudaSuccess) rc = cuda_failed();
  }
  if (rc == ATTN_OK && joined > 0) {
    cfg.gridDim = dim3((unsigned)(joined * kJoinBlocks));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, attn_window_bwd_join_kernel<D, BF16>, pk) != cudaSuccess) rc = cuda_failed();
  }
  if (cudaFreeAsync(ws, stream) != cudaSuccess) rc = cuda_failed();
  return rc;
}

}  // namespace

extern "C" {

int attn_fwd_window(const void* q, const void* k, const void* v, void* out, float* lse, int B, int H, int Hkv, int Nq,
                    int Nk, int d, int window, int sinks, float scale, int dtype, attn_stream_t stream) {
  if (int rc = check_window(q, k, v, B, H, Hkv, Nq, Nk, d, window, sinks, scale, dtype)) return rc;
  if (!out || host_misaligned(out, 16) || (lse && host_misaligned(lse, 4))) return ATTN_ERR_INVALID_ARG;
  const size_t qb = (size_t)B * Nq * H * d * 2, kb = (size_t)B * Nk * Hkv * d * 2, lb = (size_t)B * H * Nq * 4;
  const HostSpan outs[] = {{out, qb}, {lse, lb}}, ins[] = {{q, qb}, {k, kb}, {v, kb}};
  if (host_outputs_overlap(outs, 2, ins, 3)) return ATTN_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (int rc = host_device(&dev)) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool few = (long long)Nq * (H / Hkv) <= kSplitRows;
  return by_type(d, dtype, [&](auto dim, auto bf16) {
    constexpr int D = dim();
    constexpr bool BF16 = bf16();
    if (!few)
      return launch_window_fwd<D, BF16>(dev, q, k, v, out, lse, B, H, Hkv, Nq, Nk, window, sinks, scale, st);
    SplitParams p{};
    if (int rc = host_encode_bnhd(&p.tm_k, k, B, Nk, Hkv, D, dtype, 16)) return rc;
    if (int rc = host_encode_bnhd(&p.tm_v, v, B, Nk, Hkv, D, dtype, 16)) return rc;
    p.q = q; p.out = out; p.lse = lse; p.status = dev.status_ptr;
    p.B = B; p.H = H; p.Hkv = Hkv; p.Lq = Nq; p.Nk = Nk; p.causal = 1; p.window = window; p.sinks = sinks;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.timeout_ns = host_timeout_ns();
    p.inject = host_inject();
    return launch_split_rows<D, BF16, false>(dev, p, st);
  });
}

int attn_bwd_window(const void* q, const void* k, const void* v, const void* o, const long long* o_strides,
                    const void* dout, const float* lse, void* dq, void* dk, void* dv, int B, int H, int Hkv, int Nq,
                    int Nk, int d, int window, int sinks, float scale, int dtype, attn_stream_t stream) {
  if (int rc = check_window(q, k, v, B, H, Hkv, Nq, Nk, d, window, sinks, scale, dtype)) return rc;
  if (!o || !dout || !lse || !dq || !dk || !dv) return ATTN_ERR_INVALID_ARG;
  if (host_misaligned(o, 16) || host_misaligned(dout, 16) || host_misaligned(lse, 4) || host_misaligned(dq, 16) ||
      host_misaligned(dk, 16) || host_misaligned(dv, 16))
    return ATTN_ERR_INVALID_ARG;
  const size_t qb = (size_t)B * Nq * H * d * 2, kb = (size_t)B * Nk * Hkv * d * 2, lb = (size_t)B * H * Nq * 4;
  const long long strides[3] = {o_strides ? o_strides[0] : (long long)Nq * H * d, o_strides ? o_strides[1] : (long long)H * d,
                                o_strides ? o_strides[2] : d};
  long long o_last = d;  // elements that o spans
  const int o_sizes[3] = {B, Nq, H};
  for (int i = 0; i < 3; ++i) {
    if (strides[i] < 0 || strides[i] % 8 != 0 || strides[i] >= (1LL << 40)) return ATTN_ERR_INVALID_ARG;
    o_last += strides[i] * (o_sizes[i] - 1);
  }
  const HostSpan outs[] = {{dq, qb}, {dk, kb}, {dv, kb}};
  const HostSpan ins[] = {{q, qb}, {k, kb}, {v, kb}, {o, (size_t)o_last * 2}, {dout, qb}, {lse, lb}};
  if (host_outputs_overlap(outs, 3, ins, 6)) return ATTN_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (int rc = host_device(&dev)) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return by_type(d, dtype, [&](auto dim, auto bf16) {
    return launch_window_bwd<dim(), bf16()>(dev, q, k, v, o, strides, dout, lse, dq, dk, dv, B, H, Hkv, Nq, Nk, window,
                                            sinks, scale, st);
  });
}

int attn_cache_write_q4(const void* k, const void* v, void* cache, const int* block_table, const int* seq_lens,
                        const int* new_lens, int B, int Ln, int Hkv, int d, int num_blocks, int page_size,
                        int max_blocks, int dtype, attn_stream_t stream) {
  if (!k || !v || Ln <= 0) return ATTN_ERR_INVALID_ARG;
  if (int rc = check_q4(cache, block_table, seq_lens, B, Hkv, d, num_blocks, page_size, max_blocks)) return rc;
  if (!dtype_ok(dtype)) return ATTN_ERR_UNSUPPORTED;
  if (host_misaligned(k, 16) || host_misaligned(v, 16) || (new_lens && host_misaligned(new_lens, 4)))
    return ATTN_ERR_INVALID_ARG;
  const long long rows = (long long)B * Ln * Hkv;
  if (rows >= (1LL << 31) || B > kMaxGridY) return ATTN_ERR_INVALID_ARG;
  const size_t kb = (size_t)rows * d * 2;
  const HostSpan outs[] = {{cache, q4_bytes(Hkv, d, num_blocks, page_size)}};
  const HostSpan ins[] = {{k, kb}, {v, kb}, {block_table, (size_t)B * max_blocks * 4}, {seq_lens, (size_t)B * 4},
                          {new_lens, (size_t)B * 4}};
  if (host_outputs_overlap(outs, 1, ins, 5)) return ATTN_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (int rc = host_device(&dev)) return rc;
  const Q4WriteParams p{k, v, static_cast<uint8_t*>(cache), block_table, seq_lens, new_lens, dev.status_ptr,
                        B, Ln, Hkv, num_blocks, page_size, max_blocks};
  return by_type(d, dtype, [&](auto dim, auto bf16) {
    constexpr int D = dim();
    constexpr bool BF16 = bf16();
    q4_write_kernel<D, BF16><<<dim3((Ln + 7) / 8, B), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    return launched();
  });
}

int attn_cache_read_q4(const void* cache, const int* block_table, const int* seq_lens, void* k, void* v, int B,
                       int Nmax, int Hkv, int d, int num_blocks, int page_size, int max_blocks, int dtype,
                       attn_stream_t stream) {
  if (!k || !v || Nmax <= 0) return ATTN_ERR_INVALID_ARG;
  if (int rc = check_q4(cache, block_table, seq_lens, B, Hkv, d, num_blocks, page_size, max_blocks)) return rc;
  if (!dtype_ok(dtype)) return ATTN_ERR_UNSUPPORTED;
  if (host_misaligned(k, 16) || host_misaligned(v, 16)) return ATTN_ERR_INVALID_ARG;
  if ((long long)B * Nmax * Hkv >= (1LL << 31) || B > kMaxGridY) return ATTN_ERR_INVALID_ARG;
  const size_t kb = (size_t)B * Nmax * Hkv * d * 2;
  const HostSpan outs[] = {{k, kb}, {v, kb}};
  const HostSpan ins[] = {{cache, q4_bytes(Hkv, d, num_blocks, page_size)}, {block_table, (size_t)B * max_blocks * 4},
                          {seq_lens, (size_t)B * 4}};
  if (host_outputs_overlap(outs, 2, ins, 3)) return ATTN_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (int rc = host_device(&dev)) return rc;
  const Q4ReadParams p{static_cast<const uint8_t*>(cache), block_table, seq_lens, k, v, B, Nmax, Hkv, num_blocks,
                       page_size, max_blocks};
  return by_type(d, dtype, [&](auto dim, auto bf16) {
    constexpr int D = dim();
    constexpr bool BF16 = bf16();
    constexpr int rows = 8 * kQ4ReadRows;  // of a block
    q4_read_kernel<D, BF16><<<dim3((Nmax + rows - 1) / rows, B), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    return launched();
  });
}

int attn_fwd_paged_q4(const void* q, const void* cache, const int* block_table, const int* seq_lens, void* out,
                      float* lse, int B, int H, int Hkv, int Lq, int d, int num_blocks, int page_size, int max_blocks,
                      int causal, int window, int sinks, float scale, int dtype, attn_stream_t stream) {
  if (!q || !out) return ATTN_ERR_INVALID_ARG;
  if (int rc = check_q4(cache, block_table, seq_lens, B, Hkv, d, num_blocks, page_size, max_blocks)) return rc;
  if (H <= 0 || H % Hkv != 0 || Lq < 1 || Lq > 16 || (causal != 0 && causal != 1) || window < 0 || sinks < 0 ||
      !std::isfinite(scale))
    return ATTN_ERR_INVALID_ARG;
  // a window is counted back from each token's own position
  if (window > 0 && !causal && Lq > 1) return ATTN_ERR_INVALID_ARG;
  if (!dtype_ok(dtype)) return ATTN_ERR_UNSUPPORTED;
  if (host_misaligned(q, 16) || host_misaligned(out, 16) || (lse && host_misaligned(lse, 4)))
    return ATTN_ERR_INVALID_ARG;
  if ((long long)B * Lq * H >= (1LL << 31)) return ATTN_ERR_INVALID_ARG;
  const size_t qb = (size_t)B * Lq * H * d * 2;
  const HostSpan outs[] = {{out, qb}, {lse, (size_t)B * H * Lq * 4}};
  const HostSpan ins[] = {{q, qb}, {cache, q4_bytes(Hkv, d, num_blocks, page_size)},
                          {block_table, (size_t)B * max_blocks * 4}, {seq_lens, (size_t)B * 4}};
  if (host_outputs_overlap(outs, 2, ins, 4)) return ATTN_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (int rc = host_device(&dev)) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  SplitParams p{};
  p.cache = static_cast<const uint8_t*>(cache); p.block_table = block_table; p.seq_lens = seq_lens;
  p.q = q; p.out = out; p.lse = lse; p.status = dev.status_ptr;
  p.B = B; p.H = H; p.Hkv = Hkv; p.Lq = Lq; p.Nk = max_blocks * page_size;
  p.causal = causal; p.window = window; p.sinks = sinks;
  p.num_blocks = num_blocks; p.page_size = page_size; p.max_blocks = max_blocks;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.timeout_ns = host_timeout_ns();
  p.inject = host_inject();
  return by_type(d, dtype, [&](auto dim, auto bf16) { return launch_split_rows<dim(), bf16(), true>(dev, p, st); });
}

}  // extern "C"
