// block_norm_launch.cuh -- host side of block_norm.cuh: which kernel a call gets.
#pragma once

#include <algorithm>

#include "block_norm.cuh"

namespace rarn {
namespace block {

template <typename T, typename TR>
cudaError_t launch_block(const Params &p, bool vec, int num_sms, bool pdl, cudaStream_t st) {
    const int threads = p.H >= 1024 ? 1024 : (p.H + 31) / 32 * 32;
    const unsigned grid = (unsigned)std::min<int64_t>(p.T, (int64_t)num_sms * (2048 / threads));
    return launch_kernel(k_block_any<T, TR>, dim3(grid), dim3(threads), 0, st, pdl, 1, p);
}

}  // namespace block
}  // namespace rarn
