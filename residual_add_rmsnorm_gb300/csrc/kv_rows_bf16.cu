// kv_rows_bf16.cu -- per-head norm, rotation, cache write and read instantiated for __nv_bfloat16.
#include "kv_rows_launch.cuh"

namespace rarn {
namespace kv {
template cudaError_t launch_head_rows<__nv_bfloat16>(const RowParams &, bool, int, bool, cudaStream_t);
template cudaError_t launch_cache_read<__nv_bfloat16>(const ReadParams &, int, int, bool, cudaStream_t);
}  // namespace kv
}  // namespace rarn
