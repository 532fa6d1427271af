// One product kernel's launch, shared by the launchers' translation units.
#pragma once

#include "launch.h"
#include "linear.cuh"

namespace da {

template <int CG, bool A_MN, bool B_MN, int EPI>
cudaError_t launch_linear_cg(const LinearParams& p, int grid, cudaStream_t s) {
  using C = LinearCfg<CG, A_MN, B_MN, EPI>;
  auto kernel = linear_kernel<CG, A_MN, B_MN, EPI>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(C::NTHREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool A_MN, bool B_MN, int EPI>
cudaError_t launch_linear_as(const LinearParams& p, int cg, int grid, cudaStream_t s) {
  return cg == 2 ? launch_linear_cg<2, A_MN, B_MN, EPI>(p, grid, s) : launch_linear_cg<1, A_MN, B_MN, EPI>(p, grid, s);
}

}  // namespace da
