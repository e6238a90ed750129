// Launches that depend on the one before them in the stream: the kernel may
// start while its predecessor drains, and waits for the predecessor's results
// in grid_dependency_wait().
#pragma once

#include <cuda_runtime.h>

#include <functional>
#include <mutex>
#include <new>
#include <unordered_map>
#include <utility>

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
// lock and the limit only grows.  The library has some 150 such kernels, and a table
// has an entry for each device: it grows with them.
inline cudaError_t prepare_kernel(const void* kernel, int smem, int* regs = nullptr) {
  struct Entry { int smem, regs; };
  struct Hash {
    size_t operator()(const std::pair<const void*, int>& k) const {
      return std::hash<const void*>()(k.first) + 0x9e3779b9u * (size_t)k.second;
    }
  };
  static std::mutex lock;
  static auto* const table = new std::unordered_map<std::pair<const void*, int>, Entry, Hash>;  // (lives as long as the process)
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  try {
    std::lock_guard<std::mutex> held(lock);
    const auto key = std::make_pair(kernel, device);
    auto at = table->find(key);
    if (at == table->end()) {
      cudaFuncAttributes fa;
      e = cudaFuncGetAttributes(&fa, kernel);
      if (e != cudaSuccess) return e;
      at = table->emplace(key, Entry{-1, fa.numRegs}).first;
    }
    if (smem > at->second.smem) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      at->second.smem = smem;
    }
    if (regs) *regs = at->second.regs;
    return cudaSuccess;
  } catch (const std::bad_alloc&) {
    return cudaErrorMemoryAllocation;
  }
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
