// The dynamic shared memory that a kernel may be launched with: a setting of the
// kernel on one device, made at its first launch there (0.4 us a call otherwise).
// Two host threads that both make it make the same one.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace gp {

template <auto kernel>
cudaError_t allow_shared(int bytes) {
  static std::atomic<uint64_t> made{0};  // a bit a device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (made.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) made.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace gp
