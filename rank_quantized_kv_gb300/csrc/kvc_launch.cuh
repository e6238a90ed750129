// Launches that depend on the one before them in the stream: the kernel may
// start while its predecessor drains, and waits for the predecessor's results
// in grid_dependency_wait().
#pragma once

#include <cuda_runtime.h>

namespace kvc {

// Until every launch that this one depends on has finished and its writes are
// visible.  (Nothing to wait for in an ordinary launch.)
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The dependent launch may start once every block has called this or exited.
__device__ __forceinline__ void grid_dependents_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Attributes of a kernel on the current device, asked for once per thread: its
// registers, and the dynamic shared memory that it may use raised to `smem`.
// (Both calls take about a microsecond, which a decode step notices.)
inline cudaError_t prepare_kernel(const void* kernel, int smem, int* regs = nullptr) {
  struct Entry { const void* kernel; int device, smem, regs; };
  thread_local Entry cache[64];
  thread_local int n = 0;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  Entry* at = nullptr;
  for (int i = 0; i < n; ++i)
    if (cache[i].kernel == kernel && cache[i].device == device) at = &cache[i];
  Entry fresh{kernel, device, -1, 0};
  if (!at) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    fresh.regs = fa.numRegs;
    at = n < 64 ? &(cache[n++] = fresh) : &fresh;
  }
  if (smem > at->smem) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    at->smem = smem;
  }
  if (regs) *regs = at->regs;
  return cudaSuccess;
}

template <class... Params, class... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem,
                             cudaStream_t stream, const Args&... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace kvc
