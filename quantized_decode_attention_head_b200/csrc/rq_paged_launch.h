// Launches of the paged kernels: dynamic shared memory enabled once per device
// and kernel, programmatic dependent launch.
//
// Ordering.  The first kernel of a call waits for the stream's earlier work
// (griddepcontrol.wait) before it reads anything, and only then lets its
// dependents start.  So a later kernel of the same call may read what the
// caller passed (lengths, tables, pages, queries) at once, and waits only
// before it touches what an earlier kernel of the call writes; every kernel
// waits before it ends, so that the completion of the last one covers all.
#pragma once

#include <atomic>

#include <cuda_runtime.h>

namespace rq {

template <auto Kernel, class... Args>
cudaError_t launch_pdl(dim3 grid, int threads, int smem, cudaStream_t s, const Args&... args) {
  constexpr int kDevices = 64;
  static std::atomic<bool> ready[kDevices];  // per kernel
  if (smem > 48 * 1024) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices || !ready[dev].load(std::memory_order_acquire)) {
      e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      if (dev < kDevices) ready[dev].store(true, std::memory_order_release);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, Kernel, args...);
}

}  // namespace rq
