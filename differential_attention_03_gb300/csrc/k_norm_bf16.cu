// The norms around a block: bf16 rows and stream.
#include "norm_launch.cuh"

namespace da {

cudaError_t launch_norm_bf16(const NormParams& p, const NormShape& h, bool grad, int grid, int smem, cudaStream_t s) {
  return launch_norm_types<__nv_bfloat16, __nv_bfloat16>(p, h, grad, grid, smem, s);
}

}  // namespace da
