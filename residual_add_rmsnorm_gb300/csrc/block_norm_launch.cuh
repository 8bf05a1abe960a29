// block_norm_launch.cuh -- host side of block_norm.cuh: which kernel a call gets.
#pragma once

#include <algorithm>

#include "block_norm.cuh"

namespace rarn {
namespace block {

template <typename T, typename TR, int VPT, bool kWarp, bool kPipe>
cudaError_t launch_vec(const Params &p, int num_sms, int threads, bool pdl, cudaStream_t st) {
    // every CTA has the same number of rounds or one less
    const int per = kWarp ? threads / 32 : 1;
    const int64_t slots = (int64_t)num_sms * std::max(1, 2048 / threads);
    const int64_t ctas = (p.T + per - 1) / per, rounds = (ctas + slots - 1) / slots;
    const dim3 grid((unsigned)((ctas + rounds - 1) / rounds));
    return p.gate ? launch_kernel(k_block_vec<T, TR, VPT, true, kWarp, kPipe>, grid, dim3(threads),
                                  0, st, pdl, 1, p)
                  : launch_kernel(k_block_vec<T, TR, VPT, false, kWarp, kPipe>, grid,
                                  dim3(threads), 0, st, pdl, 1, p);
}

// Rows that an SM holds side by side without the next row's registers (800 threads
// of 80) need no next row: 517 rows of 5120, binary32 residual, gates, 11.2 -> 10.1 us.
constexpr int kSideBySide = 800;

template <typename T, typename TR, int VPT>
cudaError_t launch_cta(const Params &p, int num_sms, bool pdl, cudaStream_t st) {
    const int n = p.H / DT<T>::EPV, threads = ((n + VPT - 1) / VPT + 31) / 32 * 32;
    return p.T <= (int64_t)num_sms * (kSideBySide / threads)
               ? launch_vec<T, TR, VPT, false, false>(p, num_sms, threads, pdl, st)
               : launch_vec<T, TR, VPT, false, true>(p, num_sms, threads, pdl, st);
}

template <typename T, typename TR>
cudaError_t launch_block(const Params &p, bool vec, int num_sms, bool pdl, cudaStream_t st) {
    const int n = p.H / DT<T>::EPV;  // packs
    if (vec && n <= 128) {
        if (n <= 32) return launch_vec<T, TR, 1, true, true>(p, num_sms, 256, pdl, st);
        if (n <= 64) return launch_vec<T, TR, 2, true, true>(p, num_sms, 256, pdl, st);
        return launch_vec<T, TR, 4, true, true>(p, num_sms, 256, pdl, st);
    }
    if (vec && n <= 4096) {
        // about 256 threads a row (16384 rows of 5120: 111 us with four packs a thread, 130
        // with two), or as many as there are packs where a row has an SM for itself
        const int target = p.T <= num_sms ? 1024 : 256;
        if (n <= target) return launch_cta<T, TR, 1>(p, num_sms, pdl, st);
        if (n <= 2 * target && n <= 1024) return launch_cta<T, TR, 2>(p, num_sms, pdl, st);
        if (n <= 2048) return launch_cta<T, TR, 4>(p, num_sms, pdl, st);
        return launch_vec<T, TR, 8, false, false>(p, num_sms, (n + 255) / 256 * 32, pdl, st);
    }
    // single elements: 8 or 16 to a thread while a row fits 512 threads
    auto any = [&](auto kernel, int each, int most) {
        const int threads = std::min(most, ((p.H + each - 1) / each + 31) / 32 * 32);
        const int64_t slots = (int64_t)num_sms * (2048 / threads);
        const int64_t rounds = (p.T + slots - 1) / slots;
        return launch_kernel(kernel, dim3((unsigned)((p.T + rounds - 1) / rounds)), dim3(threads),
                             0, st, pdl, 1, p);
    };
    if (p.H <= 8 * 512) return any(k_block_any<T, TR, 8>, 8, 512);
    if (p.H <= 16 * 512) return any(k_block_any<T, TR, 16>, 16, 512);
    return any(k_block_any<T, TR, 0>, 1, 1024);
}

}  // namespace block
}  // namespace rarn
