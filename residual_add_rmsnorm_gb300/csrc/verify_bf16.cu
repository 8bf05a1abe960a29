// verify_bf16.cu -- verification of drafted tokens, probabilities in __nv_bfloat16.
#include "verify_launch.cuh"

namespace rarn {
namespace verify {
template cudaError_t launch_verify<__nv_bfloat16>(const Params &, int, bool, cudaStream_t);
}  // namespace verify
}  // namespace rarn
