// launch.h -- kernel launches that may start while the kernel before them on the stream still runs.
#pragma once
#include <cuda_runtime.h>

#include <atomic>

namespace sdpa {

// Launches kern(args...).  early: with programmatic stream serialization, so the grid may be set up
// once every block of the kernel before it has called grid_launch_dependents() or ended; the
// kernel itself waits with grid_wait() (ptx.cuh).  0, or -1 on a launch error.
template <class... P, class... A>
inline int launch_kernel(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, bool early,
                         const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, P(args)...) == cudaSuccess ? 0 : -1;
}

// Allows a kernel its dynamic shared memory, once a device (a bit for each in the kernel's own word).
template <auto KERN>
inline bool allow_smem(int bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (done.load(std::memory_order_acquire) >> dev & 1ull) return true;
  if (cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done.fetch_or(1ull << dev, std::memory_order_acq_rel);
  return true;
}

}  // namespace sdpa
