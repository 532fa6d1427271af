// Tree decode, V2 at d = 128, in the three cache formats.
#include "tree_launch.cuh"

namespace da {

cudaError_t launch_tree_v2_d128(const TreeParams& p, int fmt, cudaStream_t s) {
  if (fmt == kCacheBf16) return launch_tree<128, true, kCacheBf16>(p, s);
  if (fmt == kCacheFp8k) return launch_tree<128, true, kCacheFp8k>(p, s);
  return launch_tree<128, true, kCacheFp8>(p, s);
}

}  // namespace da
