// Launchers of the products for few tokens.
#include "launch.h"
#include "linear_few.cuh"

namespace da {

namespace {

template <bool W_MN, int EPI>
cudaError_t launch_few_as(const LinearParams& p, int grid, int smem_bytes, cudaStream_t s) {
  auto kernel = linear_few_kernel<W_MN, EPI>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewMaxSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = smem_bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cs;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cs > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t linear_few_clusters(int cs, int* n) {
  auto kernel = linear_few_kernel<false, kEpiBf16>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewMaxSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = kFewMaxSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(n, kernel, &cfg);
}

cudaError_t launch_linear_few(const LinearParams& p, int epi, bool w_mn, int grid, int smem_bytes, cudaStream_t s) {
  if (w_mn) return launch_few_as<true, kEpiBf16>(p, grid, smem_bytes, s);
  switch (epi) {
    case kEpiGated: return launch_few_as<false, kEpiGated>(p, grid, smem_bytes, s);
    case kEpiF32: return launch_few_as<false, kEpiF32>(p, grid, smem_bytes, s);
    default: return launch_few_as<false, kEpiBf16>(p, grid, smem_bytes, s);
  }
}

}  // namespace da
