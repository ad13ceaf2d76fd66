#include "ol_tree.cuh"
namespace ol {
bool fast_tree_supported(const TreeParams&) { return false; }
cudaError_t launch_fast_tree(TreeParams&, int, cudaStream_t) { return cudaErrorNotSupported; }
}  // namespace ol
