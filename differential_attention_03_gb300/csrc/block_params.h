// Parameter blocks of the element-wise backward kernels of the products
// (act_grad.cuh), of the norms around a block (residual_norm.cuh) and of the
// fixed-order sums over partial rows that both end in.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace da {

constexpr int kNormMaxD = 8192;
constexpr int kNormMaxSmem = 224 * 1024;
constexpr int kNormMaxStages = 8;
// Layouts of a row (residual_norm.cuh).
enum NormLayout { kSubWarp, kRing, kPlain, kPlainWarp };

struct ActGradParams {
  const __nv_bfloat16* dy;   // [M, N] (gated: dh [M, N])
  const __nv_bfloat16* pre;  // [M, N]; gated: [M, 2 N]; nullptr without an activation
  __nv_bfloat16* dz;         // [M, N]; gated: [M, 2 N]; nullptr: column sums alone
  float* part;               // [chunks][N] column sums or nullptr
  long long ldy, ldp, ldz;
  int M, N, act, chunks;     // chunks: of rows (gridDim.y)
};

// dst[j] = sum_c part[c][j] for up to three tensors at once, in a fixed order: every 32nd row by one warp, these 32 sums in
// a butterfly.
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
  const float* gate;     // [gate_rows, D] or nullptr
  const float *gamma_post, *gamma;  // [D] or nullptr: ones
  void *s_out, *y_out;              // forward; either may be nullptr
  void *dx, *dresidual;             // backward; either may be nullptr
  float *part_gamma, *part_post;    // [CTAs][D] or nullptr
  float* part_gate;                 // [chunks][groups][D]; dgate itself with one chunk, or a gate a row; nullptr: not wanted
  long long rows, gate_rows;
  // Rows that share a gate row (forward).  Backward: groups of rows that are summed over together (with a gate a row: all
  // rows are one group), in `chunks` pieces of chunk_rows rows; pieces = groups * chunks.
  long long groups, group_rows, chunk_rows, pieces;
  int chunks;
  int D;
  int lanes;   // lanes that share a row (kSubWarp, kPlainWarp)
  int stages;  // rows on their way (kRing)
  int off_combined;  // where gamma_post times the gate lies in shared memory (backward, kRing of 16 elements a thread; -1: nowhere)
  int off_post;  // where the sums for dgamma_post lie in shared memory (backward): D floats, or D a worker of the CTA
  float scale, eps;
  int post, norm;  // whether x is normed, whether y is wanted or given
  int* status;
};

// How a row is laid over threads: `nv` vectors of `vec` elements a thread; layout: NormLayout.
struct NormShape {
  int vec, nv, threads, layout, lanes;
};

}  // namespace da
