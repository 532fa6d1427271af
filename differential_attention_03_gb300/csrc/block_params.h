// Parameter blocks of the element-wise backward kernels of the products
// (act_grad.cuh), of the norms around a block (residual_norm.cuh) and of the
// fixed-order sums over partial rows that both end in.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace da {

constexpr int kNormMaxD = 8192;

struct ActGradParams {
  const __nv_bfloat16* dy;   // [M, N] (gated: dh [M, N])
  const __nv_bfloat16* pre;  // [M, N]; gated: [M, 2 N]; nullptr without an activation
  __nv_bfloat16* dz;         // [M, N]; gated: [M, 2 N]; nullptr: column sums alone
  float* part;               // [chunks][N] column sums or nullptr
  long long ldy, ldp, ldz;
  int M, N, act, chunks;     // chunks: of rows (gridDim.y)
};

// dst[j] = sum_c part[c][j] in the order of c, for up to three tensors at once.
struct SumParts {
  const float* part[3];
  float* dst[3];
  long long width[3];
  int count[3];
};

struct NormParams {
  const void* x;         // [rows, D]
  const void* residual;  // [rows, D] or nullptr (forward)
  const void* s;         // the stored sum (backward)
  const void *dy, *ds;   // gradients of y and s, either may be nullptr (backward)
  const float* gate;     // [groups, D] or nullptr
  const float *gamma_post, *gamma;  // [D] or nullptr: ones
  void *s_out, *y_out;              // forward; either may be nullptr
  void *dx, *dresidual;             // backward; either may be nullptr
  float *part_gamma, *part_post;    // [workers][D] or nullptr
  float* part_gate;                 // [chunks][groups][D], or dgate itself with one chunk; nullptr: not wanted
  long long rows;
  long long group_rows;  // rows that share a row of `gate`
  long long groups;
  long long chunk_rows;  // rows of a worker's piece of a group (backward)
  long long pieces;      // groups * chunks (backward)
  int chunks;
  int D;
  float scale, eps;
  int post, norm;        // whether x is normed, whether y is wanted or given
};

// How a row is laid over threads: `nv` vectors of `vec` elements each; warp: a warp a row.
struct NormShape {
  int vec, nv, threads;
  bool warp;
};

}  // namespace da
