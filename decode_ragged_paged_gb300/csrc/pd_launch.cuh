// pd_launch.cuh -- a kernel's dynamic shared memory, allowed once per device.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace pd {

// Allows Kernel `bytes` of dynamic shared memory on the current device. The
// runtime takes about a microsecond for it, so later calls only look it up.
template <auto Kernel>
inline cudaError_t allow_smem(size_t bytes) {
  static std::atomic<bool> allowed[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < 64;
  if (known && allowed[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && known) allowed[dev].store(true, std::memory_order_release);
  if (e != cudaSuccess) cudaGetLastError();  // (the caller returns it)
  return e;
}

}  // namespace pd
