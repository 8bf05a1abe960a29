// block_norm_f16.cu -- the norms around a block for __half.
#include "block_norm_launch.cuh"

namespace rarn {
namespace block {
template cudaError_t launch_block<__half, __half>(const Params &, bool, int, bool, cudaStream_t);
template cudaError_t launch_block<__half, float>(const Params &, bool, int, bool, cudaStream_t);
}  // namespace block
}  // namespace rarn
