// The windowed attention's tensor-core kernels for jobs of 32 rows (a file of its own, to
// compile beside the others).
#include "kvc_window_mma_main.cuh"

namespace kvc {

WindowKernel window_kernel_32(const Params& kp, const Params& vp, int NCk, int* tables) {
  return mma_kernel_for<4, false>(kp, vp, NCk, tables);
}

}  // namespace kvc
