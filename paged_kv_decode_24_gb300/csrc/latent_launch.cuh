// Host-side launch of the latent attention, rotary append and differential
// attention kernels.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace pa {

// SMs of the current device, read once per device (0: unknown).
inline int sm_count() {
  static std::atomic<int> sms[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) {
    n = sms[dev & 63].load(std::memory_order_relaxed);
    if (n <= 0 && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
      sms[dev & 63].store(n, std::memory_order_relaxed);
  }
  (void)cudaGetLastError();
  return n > 0 ? n : 0;
}

// Launch kern(args...) on `grid` CTAs of `threads` threads with `smem` bytes
// of dynamic shared memory, allowing programmatic dependent launch after the
// previous kernel in the stream.  The shared-memory limit is raised once per
// device; `configured` is the instance's own bit set of configured devices.
template <typename Kernel, typename... Args>
cudaError_t launch_latent(Kernel kern, int smem, std::atomic<unsigned long long>& configured, int grid,
                          int threads, cudaStream_t stream, const Args&... args) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (smem > 0 && !(configured.load() & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace pa
