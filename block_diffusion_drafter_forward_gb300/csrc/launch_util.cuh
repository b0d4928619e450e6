// Host-side launch helpers shared by the projection GEMM and attention launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

namespace dflash {

// Raise kernel `kern`'s dynamic shared-memory limit to `bytes` on the current device, once per
// device.  A function attribute belongs to the device's context, so a process that drives
// several GPUs sets it on each; `done` holds one bit per device id below 64 (higher ids set
// it on every call, which is harmless).
template <typename K>
inline cudaError_t smem_attr_once(K kern, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

// SMs of the current device (asked once per device).
inline cudaError_t sm_count(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev >= 0 && dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
  return e;
}

// Tensor map over rows of `heads` heads (head_dim bf16 each, contiguous): boxes of 64 dims x box_heads x
// box_rows in the 128-byte swizzle.  In gemm_tc.cu, beside the other map.
bool make_tmap_heads_bf16(CUtensorMap* map, const void* base, int64_t rows, int heads, int head_dim, int64_t ld_elems,
                          int box_heads, int box_rows);

}  // namespace dflash
