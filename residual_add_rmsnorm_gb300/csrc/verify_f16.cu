// verify_f16.cu -- verification of drafted tokens, probabilities in __half.
#include "verify_launch.cuh"

namespace rarn {
namespace verify {
template cudaError_t launch_verify<__half>(const Params &, int, bool, cudaStream_t);
}  // namespace verify
}  // namespace rarn
