// No shape runs on the tensor cores yet.
#include "tree_scores_tc.cuh"
namespace msa {
bool tree_scores_tc_supported(const Dims&) { return false; }
cudaError_t launch_tree_scores_tc(const Dims&, const void*, const void*, const void*, int, float*, cudaStream_t, int*) { return cudaErrorNotSupported; }
}
