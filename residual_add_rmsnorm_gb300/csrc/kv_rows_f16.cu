// kv_rows_f16.cu -- per-head norm, rotation, cache write and read instantiated for __half.
#include "kv_rows_launch.cuh"

namespace rarn {
namespace kv {
template cudaError_t launch_head_rows<__half>(const RowParams &, bool, int, bool, cudaStream_t);
template cudaError_t launch_cache_read<__half>(const ReadParams &, int, int, bool, cudaStream_t);
}  // namespace kv
}  // namespace rarn
