// One pair of types of the norms around a block: a translation unit each, so that they compile in parallel.
// Programmatic dependents: their CTAs come up while the kernel before them ends.
#pragma once

#include "launch.h"
#include "residual_norm.cuh"

namespace da {

template <class Kernel>
cudaError_t launch_kernel(Kernel kernel, const NormParams& p, int grid, int threads, int smem, cudaStream_t s) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxSmem);
    if (e != cudaSuccess) return e;
  }
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
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename TX, typename TS>
cudaError_t launch_norm_types(const NormParams& p, const NormShape& h, bool grad, int grid, int smem, cudaStream_t s) {
  auto go = [&](auto kernel) { return launch_kernel(kernel, p, grid, h.threads, smem, s); };
  if (grad) switch (h.layout) {
      case kSubWarp: return go(residual_norm_grad_kernel<TX, TS, 8, 1, kSubWarp>);
      case kPlainWarp:
        return h.vec == 2 ? go(residual_norm_grad_kernel<TX, TS, 2, 4, kPlainWarp>) : go(residual_norm_grad_kernel<TX, TS, 1, 8, kPlainWarp>);
      case kPlain:
        if (h.vec == 2) return h.nv == 4 ? go(residual_norm_grad_kernel<TX, TS, 2, 4, kPlain>) : go(residual_norm_grad_kernel<TX, TS, 2, 8, kPlain>);
        return h.nv == 8 ? go(residual_norm_grad_kernel<TX, TS, 1, 8, kPlain>) : go(residual_norm_grad_kernel<TX, TS, 1, 16, kPlain>);
      default:
        if (h.nv == 2) return go(residual_norm_grad_kernel<TX, TS, 8, 2, kRing>);
        if (!p.norm || p.stages < 2) return go(residual_norm_grad_kernel<TX, TS, 8, 1, kRing>);
        return p.post ? go(residual_norm_grad_pairs_kernel<TX, TS, true>) : go(residual_norm_grad_pairs_kernel<TX, TS, false>);
    }
  switch (h.layout) {
    case kSubWarp: return go(residual_norm_kernel<TX, TS, 8, 1, kSubWarp>);
    case kPlainWarp: return h.vec == 2 ? go(residual_norm_kernel<TX, TS, 2, 4, kPlainWarp>) : go(residual_norm_kernel<TX, TS, 1, 8, kPlainWarp>);
    case kPlain:
      if (h.vec == 2) return h.nv == 4 ? go(residual_norm_kernel<TX, TS, 2, 4, kPlain>) : go(residual_norm_kernel<TX, TS, 2, 8, kPlain>);
      return h.nv == 8 ? go(residual_norm_kernel<TX, TS, 1, 8, kPlain>) : go(residual_norm_kernel<TX, TS, 1, 16, kPlain>);
    default: return h.nv == 1 ? go(residual_norm_kernel<TX, TS, 8, 1, kRing>) : go(residual_norm_kernel<TX, TS, 8, 2, kRing>);
  }
}

}  // namespace da
