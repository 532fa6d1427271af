// Launchers of the norms around a block.  Programmatic dependents: their CTAs come up while the kernel before them ends.
#include "launch.h"
#include "residual_norm.cuh"

namespace da {

namespace {

template <typename TX, typename TS, int VEC, int NV, int LAYOUT>
cudaError_t launch_as(const NormParams& p, bool grad, int grid, int threads, int smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto go = [&](auto kernel) {
    if (LAYOUT == kRing) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxSmem);
      if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, kernel, p);
  };
  return grad ? go(residual_norm_grad_kernel<TX, TS, VEC, NV, LAYOUT>) : go(residual_norm_kernel<TX, TS, VEC, NV, LAYOUT>);
}

template <typename TX, typename TS>
cudaError_t launch_types(const NormParams& p, const NormShape& h, bool grad, int grid, int smem, cudaStream_t s) {
  switch (h.layout) {
    case kSubWarp: return launch_as<TX, TS, 8, 1, kSubWarp>(p, grad, grid, h.threads, smem, s);
    case kPlainWarp: return launch_as<TX, TS, 1, 8, kPlainWarp>(p, grad, grid, h.threads, smem, s);
    case kPlain: return h.nv == 8 ? launch_as<TX, TS, 1, 8, kPlain>(p, grad, grid, h.threads, smem, s)
                                  : launch_as<TX, TS, 1, 16, kPlain>(p, grad, grid, h.threads, smem, s);
    default: return h.nv == 1 ? launch_as<TX, TS, 8, 1, kRing>(p, grad, grid, h.threads, smem, s)
                              : launch_as<TX, TS, 8, 2, kRing>(p, grad, grid, h.threads, smem, s);
  }
}

}  // namespace

cudaError_t launch_residual_norm(const NormParams& p, const NormShape& h, bool x_f32, bool s_f32, bool grad, int grid, int smem,
                                 cudaStream_t s) {
  if (x_f32) return launch_types<float, float>(p, h, grad, grid, smem, s);
  if (s_f32) return launch_types<__nv_bfloat16, float>(p, h, grad, grid, smem, s);
  return launch_types<__nv_bfloat16, __nv_bfloat16>(p, h, grad, grid, smem, s);
}

}  // namespace da
