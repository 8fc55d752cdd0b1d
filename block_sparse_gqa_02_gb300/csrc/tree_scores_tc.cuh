// tcgen05 index scores of drafted tokens (bf16 queries, index_dim 128, block 128).
#pragma once
#include "common.cuh"

namespace msa {
bool tree_scores_tc_supported(const Dims& p);
cudaError_t launch_tree_scores_tc(const Dims& p, const void* idx_q, const void* idx_k,
                                  const void* idx_draft, int packed, float* scores,
                                  cudaStream_t st, int* status);
}  // namespace msa
