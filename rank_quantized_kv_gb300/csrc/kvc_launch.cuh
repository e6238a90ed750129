// Launches that depend on the one before them in the stream: the kernel may
// start while its predecessor drains, and waits for the predecessor's results
// in grid_dependency_wait().
#pragma once

#include <cuda_runtime.h>

#include <mutex>

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

// Attributes of a kernel on the current device, asked for once: its registers,
// and the dynamic shared memory that it may use raised to `smem`.  (Both calls
// take about a microsecond, which a decode step notices.)  The limit belongs to
// the kernel, not to the calling thread, so all threads share one table under a
// lock and the limit only grows.
inline cudaError_t prepare_kernel(const void* kernel, int smem, int* regs = nullptr) {
  struct Entry { const void* kernel; int device, smem, regs; };
  static std::mutex lock;
  constexpr int kEntries = 512;  // (kernel, device) pairs; the library has about 30 such kernels
  static Entry cache[kEntries];
  static int n = 0;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> held(lock);
  int i = 0;
  while (i < n && (cache[i].kernel != kernel || cache[i].device != device)) ++i;
  if (i == n) {
    if (n == kEntries) return cudaErrorMemoryAllocation;
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    cache[n++] = Entry{kernel, device, -1, fa.numRegs};
  }
  if (smem > cache[i].smem) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cache[i].smem = smem;
  }
  if (regs) *regs = cache[i].regs;
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
