// Which tree-decode kernel takes a call: keys as the MMAs' rows (tree_cols.cuh: fp8 caches) or tokens (tree_rows.cuh: any).
#pragma once

#include "tree_cols.cuh"
#include "tree_rows.cuh"

namespace da {

// Row scales make keys as rows the faster one for as many rows (tokens times
// pairs) of a map as it takes: fp8, n32768, when both took them, one token: V1
// d64 B8 H16 188 us against 286, V1 d128 B8 H8 192 against 222; 32 tokens: 284
// against 325, 203 against 244 (261 and 190 by now).  Without them HBM bounds
// both, and tokens as rows, with deeper rings, comes nearer to it (bf16, one
// token: V1 d64 323 against 336, V1 d128 312 against 320).
template <int D, bool V2, int FMT>
cudaError_t launch_tree(const TreeParams& p, cudaStream_t s) {
  if constexpr (FMT == kCacheFp8) {
    if (p.R <= 32) {
      if (p.R <= 8) return launch_tree_cols<D, V2, 8>(p, s);
      if (p.R <= 16) return launch_tree_cols<D, V2, 16>(p, s);
      return launch_tree_cols<D, V2, 32>(p, s);
    }
  }
  return launch_tree_rows<D, V2, FMT>(p, s);
}

}  // namespace da
