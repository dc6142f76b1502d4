// attn_host.h -- host-side pieces of libattn.so that its translation units share: the
// device record, the time limit of bounded waits, tensor-map encoding and buffer checks.
// Internal: nothing here is exported.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "attn.h"

namespace attn_b200 {

struct DeviceInfo {
  int device;       // index of the current device
  int sm_count;
  int* status_ptr;  // the device's status word
};

// The current device's record (ATTN_ERR_UNSUPPORTED unless it is an sm_100 part).
int host_device(DeviceInfo* out);

// Limit of every bounded device wait, as attn_debug_set left it.
unsigned long long host_timeout_ns();

// Fault to inject, as attn_debug_set left it (0: none).
int host_inject();

// 4-D view (d, H, N, B) of a contiguous 16-bit [B, N, H, d] tensor; box (64, box_heads,
// box_rows, 1), 128-byte swizzle.
int host_encode_bnhd(CUtensorMap* map, const void* ptr, int B, int N, int H, int d, int dtype,
                     int box_rows, int box_heads = 1);

// What an entry point returns for a runtime call that failed.  The runtime keeps the error until it
// is read; left there, the thread's next launch would be taken for a failed one.
inline int cuda_failed() {
  cudaGetLastError();
  return ATTN_ERR_CUDA;
}

constexpr int kHostMaxDevices = 64;

// Raise a kernel's dynamic shared-memory limit, once per device.
template <auto Kernel>
int host_raise_smem(const DeviceInfo& dev, int bytes) {
  static std::atomic<bool> done[kHostMaxDevices] = {};
  if (done[dev.device].load(std::memory_order_acquire)) return ATTN_OK;
  if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return cuda_failed();
  done[dev.device].store(true, std::memory_order_release);
  return ATTN_OK;
}

inline bool host_misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

struct HostSpan {
  const void* ptr;
  size_t bytes;
};

inline bool host_overlap(const HostSpan& a, const HostSpan& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.ptr), y = reinterpret_cast<uintptr_t>(b.ptr);
  return a.ptr && b.ptr && x < y + b.bytes && y < x + a.bytes;
}

// True if a written buffer overlaps another written one or a read one (null spans are skipped).
inline bool host_outputs_overlap(const HostSpan* outs, int n_out, const HostSpan* ins, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (host_overlap(outs[i], ins[j])) return true;
    for (int j = i + 1; j < n_out; ++j)
      if (host_overlap(outs[i], outs[j])) return true;
  }
  return false;
}

}  // namespace attn_b200
