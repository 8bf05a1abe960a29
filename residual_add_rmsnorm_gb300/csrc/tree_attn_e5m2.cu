// tree_attn_e5m2.cu -- attention over an e5m2 cache.
#include "tree_attn_launch.cuh"

namespace rarn {
namespace tree {
template cudaError_t launch_tree<true>(const Params &, const Plan &, int, bool, cudaStream_t);
}  // namespace tree
}  // namespace rarn
