// block_norm_f32.cu -- the norms around a block for float.
#include "block_norm_launch.cuh"

namespace rarn {
namespace block {
template cudaError_t launch_block<float, float>(const Params &, bool, int, bool, cudaStream_t);
}  // namespace block
}  // namespace rarn
