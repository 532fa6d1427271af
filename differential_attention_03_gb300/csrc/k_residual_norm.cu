// Launchers of the norms around a block.
#include "launch.h"
#include "residual_norm.cuh"

namespace da {

namespace {

template <typename TX, typename TS, int VEC, int NV, bool kWarp>
cudaError_t launch_as(const NormParams& p, bool grad, int grid, int threads, cudaStream_t s) {
  if (grad)
    residual_norm_grad_kernel<TX, TS, VEC, NV, kWarp><<<grid, threads, 0, s>>>(p);
  else
    residual_norm_kernel<TX, TS, VEC, NV, kWarp><<<grid, threads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename TX, typename TS>
cudaError_t launch_types(const NormParams& p, const NormShape& h, bool grad, int grid, cudaStream_t s) {
  if (h.vec == 8) {
    if (h.warp) return launch_as<TX, TS, 8, 1, true>(p, grad, grid, 256, s);
    if (h.nv == 1) return launch_as<TX, TS, 8, 1, false>(p, grad, grid, h.threads, s);
    return launch_as<TX, TS, 8, 2, false>(p, grad, grid, h.threads, s);
  }
  if (h.warp) return launch_as<TX, TS, 1, 8, true>(p, grad, grid, 256, s);
  if (h.nv == 8) return launch_as<TX, TS, 1, 8, false>(p, grad, grid, h.threads, s);
  return launch_as<TX, TS, 1, 16, false>(p, grad, grid, h.threads, s);
}

}  // namespace

cudaError_t launch_residual_norm(const NormParams& p, const NormShape& h, bool x_f32, bool s_f32, bool grad, int grid,
                                 cudaStream_t s) {
  if (x_f32) return launch_types<float, float>(p, h, grad, grid, s);
  if (s_f32) return launch_types<__nv_bfloat16, float>(p, h, grad, grid, s);
  return launch_types<__nv_bfloat16, __nv_bfloat16>(p, h, grad, grid, s);
}

}  // namespace da
