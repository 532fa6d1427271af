// Launchers of the forward products (K-major operands).
#include "linear_launch.cuh"

namespace da {

cudaError_t launch_linear_fwd(const LinearParams& p, int epi, int cg, int grid, cudaStream_t s) {
  switch (epi) {
    case kEpiGated: return launch_linear_as<false, false, kEpiGated>(p, cg, grid, s);
    case kEpiF32: return launch_linear_as<false, false, kEpiF32>(p, cg, grid, s);
    default: return launch_linear_as<false, false, kEpiBf16>(p, cg, grid, s);
  }
}

}  // namespace da
