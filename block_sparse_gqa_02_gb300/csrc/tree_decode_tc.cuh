// tcgen05 attention of a tree of drafted tokens (bf16, block 128).
#pragma once
#include "common.cuh"

namespace msa {
bool tree_decode_tc_supported(const Dims& p);
int tree_decode_tc_splits(const Dims& p);
// partial outputs ws_o [B, nR, Hq, splits, d] and log-sums ws_l [B, nR, Hq, splits]
cudaError_t launch_tree_decode_tc(const Dims& p, const void* q, const void* k, const void* v,
                                  const void* k_draft, const void* v_draft, const int32_t* sel,
                                  float* ws_o, float* ws_l, cudaStream_t st, int* status);
}  // namespace msa
