// No shape runs on the tensor cores yet.
#include "tree_decode_tc.cuh"
namespace msa {
bool tree_decode_tc_supported(const Dims&) { return false; }
int tree_decode_tc_splits(const Dims&) { return 1; }
cudaError_t launch_tree_decode_tc(const Dims&, const void*, const void*, const void*, const void*, const void*, const int32_t*, float*, float*, cudaStream_t, int*) { return cudaErrorNotSupported; }
}
