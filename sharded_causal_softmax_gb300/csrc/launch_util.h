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

// Sets an attribute of `kernel` on the current device, once per device and call
// site (`done`, a static of the caller's).
template <typename K>
inline cudaError_t allow_attribute(K kernel, cudaFuncAttribute what, int value,
                                   std::atomic<bool> (&done)[kMaxCachedDevices]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool cached = dev >= 0 && dev < kMaxCachedDevices;
  if (cached && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, what, value);
  if (e == cudaSuccess && cached) done[dev].store(true, std::memory_order_release);
  return e;
}

// Allows `kernel` `bytes` of dynamic shared memory.
template <typename K>
inline cudaError_t allow_smem(K kernel, int bytes, std::atomic<bool> (&done)[kMaxCachedDevices]) {
  return allow_attribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes, done);
}

// Launches `kernel` so that its CTAs may start while the kernel before it in
// the stream still runs, if that one says so (griddepcontrol.launch_dependents);
// the kernel itself waits (griddepcontrol.wait) before it touches memory that
// kernels before it read or write.
template <typename K, typename A>
inline cudaError_t launch_early(K kernel, dim3 grid, int threads, int smem, cudaStream_t st, const A& arg) {
  cudaLaunchAttribute early = {};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, arg);
}

}  // namespace sca
