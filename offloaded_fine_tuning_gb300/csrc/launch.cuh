// Host-side helpers of the kernel launchers.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace sf {

// Reserve `bytes` of dynamic shared memory for Kern (always the same number) on
// the current device, once per kernel and device: the attribute is per device.
// Two threads that come here first set it twice, to the same value.
template <auto Kern>
bool reserve_smem(int bytes) {
  static std::atomic<uint64_t> done{0};  // a bit for each device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return false;
  }
  const uint64_t bit = uint64_t(1) << dev;
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(reinterpret_cast<const void*>(Kern), cudaFuncAttributeMaxDynamicSharedMemorySize,
                           bytes) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  done.fetch_or(bit, std::memory_order_release);
  return true;
}

// Launch `kern` so that it may be set up while the stream's previous kernel
// ends; it calls wait_primary() before it uses that kernel's results.  False
// where the launch failed; the error stays for cudaGetLastError.
template <class... P, class... A>
bool launch_dependent(void (*kern)(P...), dim3 grid, int threads, int smem, cudaStream_t st, A... args) {
  cudaLaunchAttribute after[1];
  after[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  after[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cfg.attrs = after;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...) == cudaSuccess;
}

}  // namespace sf
