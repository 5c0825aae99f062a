// Leave for a kernel to use more shared memory than 48 KB.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

namespace moe {

constexpr int kMaxKernels = 16;   // of one type, in one translation unit

// Dynamic shared memory past 48 KB has to be allowed once for a kernel and device.
template <typename K>
static bool allow_smem(K kernel, size_t smem) {
  static std::atomic<uint64_t> done[kMaxKernels];   // devices, by kernel
  static std::atomic<const void*> known[kMaxKernels];
  int dev = 0, i = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const void* id = reinterpret_cast<const void*>(kernel);
  for (; i < kMaxKernels; ++i) {
    const void* at = known[i].load(std::memory_order_acquire);
    if (at == id || (!at && known[i].compare_exchange_strong(at, id)) || at == id) break;
  }
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (i < kMaxKernels && (done[i].load(std::memory_order_acquire) & bit)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
    return false;
  if (i < kMaxKernels) done[i].fetch_or(bit, std::memory_order_release);
  return true;
}

}  // namespace moe
