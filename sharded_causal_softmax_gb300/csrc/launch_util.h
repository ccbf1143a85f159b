// Host-side launch helpers that are looked up once per device.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace sca {

constexpr int kMaxCachedDevices = 64;

// SMs of the current device.
inline int sm_count() {
  static std::atomic<int> seen[kMaxCachedDevices] = {};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
  const bool cached = dev >= 0 && dev < kMaxCachedDevices;
  if (cached && (n = seen[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();   // no device (a host-only call): leave no error behind
    return 152;
  }
  if (cached) seen[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Allows `kernel` `bytes` of dynamic shared memory on the current device,
// once per device and call site (`done`, a static of the caller's).
template <typename K>
inline cudaError_t allow_smem(K kernel, int bytes, std::atomic<bool> (&done)[kMaxCachedDevices]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool cached = dev >= 0 && dev < kMaxCachedDevices;
  if (cached && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && cached) done[dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace sca
