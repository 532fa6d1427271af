// Which tree-decode kernel takes a call: keys as the MMAs' rows (tree_cols.cuh) or tokens (tree_rows.cuh).
#pragma once

#include "tree_cols.cuh"
#include "tree_rows.cuh"

namespace da {

// Rows (tokens times pairs) of a map that the keys-as-rows kernel takes.  Row
// scales make it the faster one wherever it fits: fp8, n32768, one token: V1
// d64 B8 H16 188 us against 286, V1 d128 B8 H8 192 against 222; 32 tokens: 284
// against 325, 203 against 244.  Without them HBM bounds both up to 16 rows,
// and the tokens-as-rows kernel, with deeper rings, comes nearer to it (bf16,
// one token: V1 d64 323 against 336, V1 d128 312 against 320; 16: equal); its
// row maxima cost it at 17 to 32 (bf16 V1 d128 343 against 322, V2 184 against
// 172; at d64 358 against 372, so it keeps that).
template <int D, int FMT>
constexpr bool tree_takes_cols(int R) {
  return FMT == kCacheFp8 ? R <= 32 : (D == 128 && R > 16 && R <= 32);
}

template <int D, bool V2, int FMT>
cudaError_t launch_tree(TreeParams p, cudaStream_t s) {
  if (tree_takes_cols<D, FMT>(p.R)) {
    p.subs = p.R <= 8 ? 4 : p.R <= 16 ? 2 : 1;
    if constexpr (FMT == kCacheFp8) {
      if (p.R <= 8) return launch_tree_cols<D, V2, FMT, 8>(p, s);
      if (p.R <= 16) return launch_tree_cols<D, V2, FMT, 16>(p, s);
    }
    if constexpr (FMT == kCacheFp8 || D == 128) return launch_tree_cols<D, V2, FMT, 32>(p, s);
  }
  p.subs = p.R <= 32 ? 2 : 1;
  return launch_tree_rows<D, V2, FMT>(p, s);
}

}  // namespace da
