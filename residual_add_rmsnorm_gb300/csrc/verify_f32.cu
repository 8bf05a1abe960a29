// verify_f32.cu -- verification of drafted tokens, probabilities in float.
#include "verify_launch.cuh"

namespace rarn {
namespace verify {
template cudaError_t launch_verify<float>(const Params &, int, bool, cudaStream_t);
}  // namespace verify
}  // namespace rarn
