// Trees of drafted tokens: a token's path, position and place among the blocks (include/msa.h).
#pragma once

#include "common.cuh"

namespace msa {

using TreeWord = unsigned long long;   // bit a: drafted token a

// Path of drafted token i (mask word m) of a sequence with cache length L, 0 when the tree has no such token
// there: bits past the tree's tokens are dropped, and a token past the capacity has no place.
__device__ __forceinline__ TreeWord tree_path_of(const Dims& p, TreeWord m, int i, int L) {
  if (p.nR < 64) m &= (1ull << p.nR) - 1;
  if (!(m >> i & 1)) return 0;
  return __popcll(m) - 1 < p.Sk - L ? m : 0;               // L + depth may pass 32 bits
}

__device__ __forceinline__ TreeWord tree_path(const Dims& p, int b, int i, int L) {
  return tree_path_of(p, p.tree_mask[(size_t)b * p.nR + i], i, L);
}

// Position of a token from its path (which is not 0).
__device__ __forceinline__ int tree_pos(TreeWord path, int L) { return L + __popcll(path) - 1; }

}  // namespace msa
