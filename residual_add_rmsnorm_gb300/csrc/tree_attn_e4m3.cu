// tree_attn_e4m3.cu -- attention over an e4m3 cache.
#include "tree_attn_launch.cuh"

namespace rarn {
namespace tree {
template cudaError_t launch_tree<false>(const Params &, const Plan &, int, bool, cudaStream_t);
}  // namespace tree
}  // namespace rarn
