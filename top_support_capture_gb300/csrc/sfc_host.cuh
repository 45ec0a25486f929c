// Host-side helper of the launches: shared-memory limits, set once per kernel and device.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace sfc {

// Lets `kernel` use up to `bytes` of dynamic shared memory. `done` holds one bit per device ordinal below 64.
template <class Kernel>
cudaError_t allow_shared(Kernel kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
  return err;
}

}  // namespace sfc
