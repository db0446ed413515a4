// pd_launch.cuh -- a kernel's dynamic shared memory, allowed once per device.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace pd {

// Allows Kernel `bytes` of dynamic shared memory on the current device. The
// runtime takes about a microsecond for it, so later calls only look it up. MOST: an SM
// gives shared memory all that it can. A kernel whose CTAs have to fit side by side in calls one after
// another wants that: an SM divides its memory anew only when it is idle, and an SM that the kernel
// before left with less holds fewer of its CTAs.
template <auto Kernel, bool MOST = false>
inline cudaError_t allow_smem(size_t bytes) {
  static std::atomic<bool> allowed[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < 64;
  if (known && allowed[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && MOST)
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && known) allowed[dev].store(true, std::memory_order_release);
  if (e != cudaSuccess) cudaGetLastError();  // (the caller returns it)
  return e;
}

}  // namespace pd
