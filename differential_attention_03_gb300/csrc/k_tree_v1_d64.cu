// Tree decode, V1 at d = 64, in the three cache formats.
#include "tree_launch.cuh"

namespace da {

cudaError_t launch_tree_v1_d64(const TreeParams& p, int fmt, cudaStream_t s) {
  if (fmt == kCacheBf16) return launch_tree<64, false, kCacheBf16>(p, s);
  if (fmt == kCacheFp8k) return launch_tree<64, false, kCacheFp8k>(p, s);
  return launch_tree<64, false, kCacheFp8>(p, s);
}

}  // namespace da
