// Launchers of the backward products (one or both operands MN-major) and of
// the element-wise kernels of the backward pass.
#include "act_grad.cuh"
#include "launch.h"
#include "linear_launch.cuh"

namespace da {

cudaError_t launch_linear_dgrad(const LinearParams& p, int cg, int grid, cudaStream_t s) {
  return launch_linear_as<false, true, kEpiBf16>(p, cg, grid, s);
}

cudaError_t launch_linear_wgrad(const LinearParams& p, int epi, int cg, int grid, cudaStream_t s) {
  return epi == kEpiF32 ? launch_linear_as<true, true, kEpiF32>(p, cg, grid, s)
                        : launch_linear_as<true, true, kEpiBf16>(p, cg, grid, s);
}

namespace {
// A programmatic dependent of the kernel before it on the stream (it waits before it reads).
template <class Kernel, class Params>
cudaError_t launch_dependent(Kernel kernel, const Params& p, dim3 grid, int threads, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool kGated, int ACT>
cudaError_t launch_act_grad_as(const ActGradParams& p, cudaStream_t s) {
  return launch_dependent(act_grad_kernel<kGated, ACT>, p, dim3((p.N + 255) / 256, p.chunks), kActGradThreads, s);
}
template <bool kGated>
cudaError_t launch_act_grad_of(const ActGradParams& p, cudaStream_t s) {
  switch (p.act) {
    case DIFFATTN_ACT_RELU: return launch_act_grad_as<kGated, DIFFATTN_ACT_RELU>(p, s);
    case DIFFATTN_ACT_GELU: return launch_act_grad_as<kGated, DIFFATTN_ACT_GELU>(p, s);
    case DIFFATTN_ACT_GELU_TANH: return launch_act_grad_as<kGated, DIFFATTN_ACT_GELU_TANH>(p, s);
    case DIFFATTN_ACT_SILU: return launch_act_grad_as<kGated, DIFFATTN_ACT_SILU>(p, s);
    default: return launch_act_grad_as<kGated, DIFFATTN_ACT_NONE>(p, s);
  }
}
}  // namespace

cudaError_t launch_act_grad(const ActGradParams& p, bool gated, cudaStream_t s) {
  return gated ? launch_act_grad_of<true>(p, s) : launch_act_grad_of<false>(p, s);
}

cudaError_t launch_sum_parts(const SumParts& p, cudaStream_t s) {
  long long widest = 0;
  int n = 0;
  for (; n < 3 && p.count[n] > 0; ++n)
    if (p.width[n] > widest) widest = p.width[n];
  if (n == 0) return cudaSuccess;
  return launch_dependent(sum_parts_kernel, p, dim3(static_cast<unsigned>((widest + 31) / 32), n), 1024, s);
}

}  // namespace da
