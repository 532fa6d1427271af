// The norms around a block: fp32 rows and stream.
#include "norm_launch.cuh"

namespace da {

cudaError_t launch_norm_f32(const NormParams& p, const NormShape& h, bool grad, int grid, int smem, cudaStream_t s) {
  return launch_norm_types<float, float>(p, h, grad, grid, smem, s);
}

}  // namespace da
