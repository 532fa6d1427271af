// Parameter blocks of the product kernels (linear.cuh, linear_few.cuh) and of
// the element-wise parts of their backward pass (act.cuh), shared by the
// launchers and the host API.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace da {

// What a product kernel does with its accumulator.
constexpr int kEpiBf16 = 0;   // out = bf16(residual + act(z + bias)); pre = bf16(z + bias)
constexpr int kEpiF32 = 1;    // the same with out and residual in fp32, sums of K segments added in registers
constexpr int kEpiGated = 2;  // out = bf16(act(g) u); pre = [bf16(g) | bf16(u)]

constexpr int kLinBM = 128;   // output rows of one CTA (TMEM lanes)
constexpr int kLinBN = 256;   // accumulator columns of a tile
constexpr int kLinBK = 64;    // contraction of a ring slot (one 128-byte row)
constexpr int kLinSegBlocks = 8;  // K blocks (512 values) that one accumulator of kEpiF32 sums

constexpr int kFewMaxSmem = 232448;

// linear_few_kernel with fp32 outputs: K blocks that an accumulator of `wrows` columns sums where each segment has its own.
// A CTA has 256 columns of tensor memory (two CTAs share an SM's 512).
__host__ __device__ inline int few_segment_blocks(int blocks, int wrows) {
  const int most = 256 / wrows;
  return (blocks + most - 1) / most;
}
// Accumulators that segments of kLinSegBlocks take turns in, beside one accumulator's columns of running sums; 0: no room.
__host__ __device__ inline int few_turns(int wrows) { return 3 * wrows <= 256 ? 2 : 2 * wrows <= 256 ? 1 : 0; }

struct LinearParams {
  CUtensorMap tm_a;  // K-major: {K, M} box {64, 128}; MN-major: {M, K} box {64, 64}; 128-byte swizzle
  CUtensorMap tm_b;  // over B ({K, N} or {N, K}), box {64, 64}; linear_few: the tokens, box {64, nt}
  CUtensorMap tm_out, tm_pre;  // linear_kernel: {N, sides, M} box {128 bytes, 1, 32}; pre has two sides if gated
  const float* bias;     // [N] or nullptr
  const void* residual;  // [M, N] in the output's type or nullptr
  void* out;
  __nv_bfloat16* pre;    // [M, N] (gated [M, 2 N]) or nullptr
  long long ldr, ldo, ldp;
  int M, N, K;           // gated: N = F
  int act;
  int tiles_m, tiles_n, group_m;  // tiles_m in units of a cluster's rows
  int full;                       // tiles before the ones that come in halves
  // linear_few: features (gated: gate features) and token rows of a tile, CTAs that share its contraction, groups of
  // eight features that each of them finishes, ring slots, and where the barriers lie in shared memory
  int width, nt, cs, lg, stages, off_bars;
  int turns;  // ... whether segments of kLinSegBlocks take turns in its accumulators (few_turns)
  int* status;
};

}  // namespace da
