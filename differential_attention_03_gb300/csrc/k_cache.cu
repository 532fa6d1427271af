// Launchers of the rotary, cache append and cache keep kernels.  Each is a
// programmatic dependent of the kernel before it on the stream (it waits
// before its first global access), which hides the launch in a chain of
// short decode-step kernels.
#include "cache.cuh"
#include "cache_params.h"

namespace da {

template <class P>
static cudaError_t launch_pdl(void (*kern)(P), const P& p, dim3 grid, int threads, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_rope(const RopeParams& p, bool f32, bool vec, int gx, int gy, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy), 1);
  if (f32)
    return vec ? launch_pdl(rope_kernel<true, true>, p, grid, kRopeThreads, s)
               : launch_pdl(rope_kernel<true, false>, p, grid, kRopeThreads, s);
  return vec ? launch_pdl(rope_kernel<false, true>, p, grid, kRopeThreads, s)
             : launch_pdl(rope_kernel<false, false>, p, grid, kRopeThreads, s);
}

template <int FMT>
static cudaError_t launch_append(const AppendParams& p, dim3 grid, cudaStream_t s) {
  if (p.d == 64) return launch_pdl(cache_append_kernel<64, 128, FMT>, p, grid, kAppendThreads, s);
  return p.dv == 256 ? launch_pdl(cache_append_kernel<128, 256, FMT>, p, grid, kAppendThreads, s)
                     : launch_pdl(cache_append_kernel<128, 128, FMT>, p, grid, kAppendThreads, s);
}

cudaError_t launch_cache_append(const AppendParams& p, int gx, int gy, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy), 1);
  if (p.fmt == kCacheBf16) return launch_append<kCacheBf16>(p, grid, s);
  return p.fmt == kCacheFp8k ? launch_append<kCacheFp8k>(p, grid, s) : launch_append<kCacheFp8>(p, grid, s);
}

cudaError_t launch_cache_keep(const KeepParams& p, int gy, cudaStream_t s) {
  return launch_pdl(cache_keep_kernel, p, dim3(static_cast<unsigned>(p.B), static_cast<unsigned>(gy), 1), kKeepThreads,
                    s);
}

}  // namespace da
