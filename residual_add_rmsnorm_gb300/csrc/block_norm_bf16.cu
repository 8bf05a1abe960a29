// block_norm_bf16.cu -- the norms around a block for __nv_bfloat16.
#include "block_norm_launch.cuh"

namespace rarn {
namespace block {
template cudaError_t launch_block<__nv_bfloat16, __nv_bfloat16>(const Params &, bool, int, bool, cudaStream_t);
template cudaError_t launch_block<__nv_bfloat16, float>(const Params &, bool, int, bool, cudaStream_t);
}  // namespace block
}  // namespace rarn
