// kv_rows_launch.cuh -- host side of kv_rows.cuh: which kernel a call gets.
#pragma once

#include "kv_rows.cuh"

namespace rarn {
namespace kv {

template <typename T, int LG>
inline cudaError_t launch_head_group(const RowParams &p, int num_sms, bool pdl, cudaStream_t st) {
    const int heads = p.q.heads + p.k.heads + p.v.heads;
    constexpr int gpw = 32 / LG;
    // Several heads per group share the table's registers and keep more loads
    // in flight; one head per group gives a short call more warps.
    const int many = (heads + gpw * 4 - 1) / (gpw * 4);
    const bool wide = p.T * many >= (int64_t)num_sms * 16;
    const int chunks = wide ? many : (heads + gpw - 1) / gpw;
    const dim3 grid((unsigned)((p.T * chunks + 3) / 4));
    return wide ? launch_kernel(k_head_rows<T, LG, 4>, grid, dim3(128), 0, st, pdl, 1, p, chunks)
                : launch_kernel(k_head_rows<T, LG, 1>, grid, dim3(128), 0, st, pdl, 1, p, chunks);
}

template <typename T>
cudaError_t launch_head_rows(const RowParams &p, bool vec, int num_sms, bool pdl,
                             cudaStream_t st) {
    if (!vec) {
        const int heads = p.q.heads + p.k.heads + p.v.heads;
        return launch_kernel(k_head_rows_any<T>, dim3((unsigned)((p.T * heads + 3) / 4)),
                             dim3(128), 0, st, pdl, 1, p, heads);
    }
    const int lanes = p.D / (2 * DT<T>::EPV);
    if (lanes <= 4) return launch_head_group<T, 4>(p, num_sms, pdl, st);
    if (lanes <= 8) return launch_head_group<T, 8>(p, num_sms, pdl, st);
    if (lanes <= 16) return launch_head_group<T, 16>(p, num_sms, pdl, st);
    return launch_head_group<T, 32>(p, num_sms, pdl, st);
}

template <typename T>
cudaError_t launch_cache_read(const ReadParams &p, bool vec, bool pdl, cudaStream_t st) {
    const dim3 grid((unsigned)((p.rows + kReadRows - 1) / kReadRows));
    return vec ? launch_kernel(k_cache_read<T, true>, grid, dim3(256), 0, st, pdl, 1, p)
               : launch_kernel(k_cache_read<T, false>, grid, dim3(256), 0, st, pdl, 1, p);
}

}  // namespace kv
}  // namespace rarn
