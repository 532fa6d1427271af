// The norms around a block: bf16 rows on an fp32 stream.
#include "norm_launch.cuh"

namespace da {

cudaError_t launch_norm_mixed(const NormParams& p, const NormShape& h, bool grad, int grid, int smem, cudaStream_t s) {
  return launch_norm_types<__nv_bfloat16, float>(p, h, grad, grid, smem, s);
}

}  // namespace da
