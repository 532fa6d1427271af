// Parameter blocks of the rotary, cache and tree-decode kernels, shared with the host API.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace da {

// Rotary positions: pair i of a head turns by turns[i] 2^-64 of a full turn per position.
struct RopeTurns {
  int rot;     // rotated channels (0: none)
  int inter;   // 0: pairs (i, i + rot / 2); 1: pairs (2 i, 2 i + 1)
  float mult;  // factor on the rotated channels
  unsigned long long turns[64];
};

constexpr int kRopeThreads = 256, kRopeMaxTokens = 8;      // threads and tokens of a CTA
constexpr int kAppendThreads = 256, kAppendMaxTokens = 8;
constexpr int kKeepThreads = 256, kKeepMaxPath = 64;       // threads of a CTA, nodes of a path

struct RopeParams {
  const void* x[4];  // [B, n, heads[i], d]
  void* out[4];
  int heads[4];
  int count, head_sum;  // tensors, and the heads of all of them
  int B, n, d;
  int copy;        // some tensor is not rotated in place: its other channels are copied
  int inverse;
  int tokens_per_cta;
  unsigned magic_tok, magic_head;  // for the divisions by a token's and a head's work items (fast_div)
  const int* pos;  // [B, n], or nullptr: token t at position t
  RopeTurns rope;
};

enum : int { kCacheBf16 = 0, kCacheFp8k = 1, kCacheFp8 = 2 };

struct AppendParams {
  const __nv_bfloat16* q[2];  // [B, T, Hq, d]
  const __nv_bfloat16* k[2];  // [B, T, H, d]
  const __nv_bfloat16* v;     // [B, T, H, dv]
  __nv_bfloat16* qo[2];
  void* kc[2];                // caches [B, n, H, d], [B, n, H, dv]
  void* vc;
  float* ks[2];               // fp8: scales [B, H, n]
  float* vs;
  float kinv[2];              // fp8k: 1 / scale of each key tensor
  const int* pos;             // [B, T], or nullptr: row of the cache
  const int* lens;            // [B], or nullptr: 0
  const int* ntok;            // [B], or nullptr: T
  int B, T, Hq, H, n, d, dv, nq, nk, fmt;
  int tokens_per_cta;
  unsigned magic[3];  // for the divisions by a token's query, key and value rows (fast_div)
  RopeTurns rope;
};

struct KeepParams {
  void* base[3];  // k1, k2, v caches (k2 may be missing: count)
  float* scales[3];
  int row_bytes[3];
  int count, B, A, H, n, fmt;
  const int* lens;
  const int* path;   // [B, A]
  const int* nkeep;  // [B]
  int* new_lens;     // [B] or nullptr
};

struct TreeParams {
  CUtensorMap tm_k1;  // key caches: boxes of 128 keys x 128 bytes (e4m3 at d = 64: 64 bytes)
  CUtensorMap tm_k2;  // (V1 only)
  CUtensorMap tm_v;   // value cache: boxes of kTreeValueKeys keys x 128 bytes
  const __nv_bfloat16* q1;  // V1 [B, T, H, d]; V2 [B, T, Hq, d]
  const __nv_bfloat16* q2;  // V1 only
  const float* k1_scales;   // fp8: [B, H, n]
  const float* k2_scales;
  const float* v_scales;
  float k1_scale, k2_scale;  // fp8k
  const int* lens;           // [B], or nullptr: n - T
  const int* ntok;           // [B], or nullptr: T
  const unsigned long long* mask;  // word of (b, t) at b * mask_sb + t, or nullptr: a chain
  long long mask_sb;
  const float* lambda;      // V1
  const float* gamma;       // V1, or nullptr
  const float* lam_logits;  // V2: (b, t, pair) at b * sb + t * st + pair
  long long sb, st;
  __nv_bfloat16* out;       // V1 [B, T, H, 2 d]; V2 [B, T, Hq / 2, d]
  float scale_log2, norm_mult, eps;
  int B, T, H, n;     // H: key heads
  int pairs;          // V2: query-head pairs of a key head (V1: 1)
  int ppt;            // pairs of one row tile
  int mt;             // row tiles of a key head
  int R;              // rows of one map in a row tile: ppt * T <= 64
  int team;           // CTAs that walk the same tiles of neighbouring units side by side (divides H mt)
  int teams;          // teams the key tiles are dealt to
  int subs;           // partial states of a CTA and unit
  float* ws;
  int* status;
};

constexpr int kTreeValueKeys = 64;  // keys of a value box of the tree decode, and of a value slot of its rings

constexpr int kTreeRows = 64;  // rows of one map in a row tile of the tree decode

// Subsets of a CTA's keys that keep their own partial state: over fp8 caches tree_cols_kernel's streams, over
// fp8k ones both halves of a tile where tree_rows_kernel splits it.
__host__ __device__ constexpr int tree_subs(int fmt, int dv, int R) {
  if (fmt == kCacheFp8) return R <= 8 ? 4 : R <= 16 ? 2 : 1;
  return fmt == kCacheFp8k && dv == 128 && R <= 32 ? 2 : 1;
}
// The most of any format: what the workspace has room for.
__host__ __device__ constexpr int tree_subs_most(int R) { return R <= 8 ? 4 : R <= 32 ? 2 : 1; }

// A partial state of the tree decode: (maximum, sum) of R rows of both maps, for each subset, then their
// O from this float on (32-byte sectors), and its floats in all.
__host__ __device__ __forceinline__ size_t tree_state_o(int R, int subs) {
  return (4 * static_cast<size_t>(subs) * R + 7) & ~static_cast<size_t>(7);
}
__host__ __device__ __forceinline__ size_t tree_state_floats(int R, int subs, int dv) {
  return tree_state_o(R, subs) + 2 * static_cast<size_t>(subs) * R * dv;
}

cudaError_t launch_rope(const RopeParams& p, bool f32, bool vec, int grid_x, int grid_y, cudaStream_t s);
cudaError_t launch_cache_append(const AppendParams& p, int grid_x, int grid_y, cudaStream_t s);
cudaError_t launch_cache_keep(const KeepParams& p, int grid_y, cudaStream_t s);
cudaError_t launch_tree_v1_d64(const TreeParams& p, int fmt, cudaStream_t s);
cudaError_t launch_tree_v1_d128(const TreeParams& p, int fmt, cudaStream_t s);
cudaError_t launch_tree_v2_d128(const TreeParams& p, int fmt, cudaStream_t s);

}  // namespace da
