// kv_rows_f32.cu -- per-head norm, rotation, cache write and read instantiated for float.
#include "kv_rows_launch.cuh"

namespace rarn {
namespace kv {
template cudaError_t launch_head_rows<float>(const RowParams &, bool, int, bool, cudaStream_t);
template cudaError_t launch_cache_read<float>(const ReadParams &, int, int, bool, cudaStream_t);
}  // namespace kv
}  // namespace rarn
