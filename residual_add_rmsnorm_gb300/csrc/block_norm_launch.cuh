// block_norm_launch.cuh -- host side of block_norm.cuh: which kernel a call gets.
#pragma once

#include <algorithm>

#include "block_norm.cuh"

namespace rarn {
namespace block {

// Every CTA has the same number of rows or one less.
inline dim3 balanced(int64_t T, int num_sms, int threads, int resident = 2048) {
    const int64_t slots = (int64_t)num_sms * std::min(32, std::max(1, resident / threads));
    const int64_t rounds = (T + slots - 1) / slots;
    return dim3((unsigned)((T + rounds - 1) / rounds));
}

// With four packs a thread and the next row an SM holds 512 threads.  Rows of up to ten
// rounds of these go round by round (1000 rows of 8192: 13.0 us, in CTAs for 2048
// threads an SM, most of which wait, 16.1); more rows keep the SMs busier when a CTA that
// ends makes room for another (8192 rows of 8192: 81 us, round by round 90).  With a gate
// round by round is the better one or as good (bfloat16, one gate, without the rule and
// with it: 8192 rows of 8192 86.8 and 85.7 us, with nine gates 102.2 and 90.0, a gate a row
// 108.8 and 108.4; 16384 of 4096 83.5 and 82.7, of 5120 107.2 and 107.7, of 7168 160.5 and
// 154.6; 2000 of 16384 53.2 and 49.1, with a binary32 residual 79.5 and 69.9) but for rows
// of one warp (60000 of 1024 75.5 and 78.4, 30000 of 2048 77.4 and 75.6).
constexpr int kPipeThreads = 512, kRounds = 10;

inline dim3 piped(int64_t T, bool gate, int num_sms, int threads) {
    const int64_t slots = (int64_t)num_sms * std::min(32, std::max(1, kPipeThreads / threads));
    return balanced(T, num_sms, threads, gate || T <= kRounds * slots ? kPipeThreads : 2048);
}

template <typename T, typename TR, int VPT, bool kPipe>
cudaError_t launch_vec(const Params &p, int num_sms, int threads, bool pdl, cudaStream_t st) {
    // no thread without a pack: no bounds to check (8192 rows of 8192: 86 -> 82 us)
    const bool full = p.H / DT<T>::EPV == VPT * threads && threads <= kMaxThreads<VPT, kPipe, true>;
    const dim3 grid = kPipe && VPT == 4 ? piped(p.T, p.gate != nullptr, num_sms, threads)
                                        : balanced(p.T, num_sms, threads);
    auto go = [&](auto kernel) {
        return launch_kernel(kernel, grid, dim3(threads), 0, st, pdl, 1, p);
    };
    if (p.gate)
        return full ? go(k_block_vec<T, TR, VPT, true, kPipe, true>)
                    : go(k_block_vec<T, TR, VPT, true, kPipe, false>);
    return full ? go(k_block_vec<T, TR, VPT, false, kPipe, true>)
                : go(k_block_vec<T, TR, VPT, false, kPipe, false>);
}

// Rows that an SM holds side by side without the next row's registers (640 threads of
// 102) need no next row: 517 rows of 5120, binary32 residual, gates, 10.1 -> 7.3 us.
constexpr int kSideBySide = 640;

template <typename T, typename TR, int VPT>
cudaError_t launch_cta(const Params &p, int num_sms, bool pdl, cudaStream_t st) {
    const int n = p.H / DT<T>::EPV, threads = ((n + VPT - 1) / VPT + 31) / 32 * 32;
    return p.T <= (int64_t)num_sms * (kSideBySide / threads)
               ? launch_vec<T, TR, VPT, false>(p, num_sms, threads, pdl, st)
               : launch_vec<T, TR, VPT, true>(p, num_sms, threads, pdl, st);
}

template <typename T, typename TR>
cudaError_t launch_block(const Params &p, bool vec, int num_sms, bool pdl, cudaStream_t st) {
    const int n = p.H / DT<T>::EPV;  // packs
    if (vec && n <= 4096) {
        // As many threads as packs where a row has an SM for itself; otherwise four packs a
        // thread, also where a warp then has a row (16384 rows of 4096: 81 us, with two
        // packs 101; 30000 of 1024: 38.8, with a row to a warp of eight 44).
        if (n <= 32 || (p.T <= num_sms && n <= 1024))
            return launch_cta<T, TR, 1>(p, num_sms, pdl, st);
        if (n <= 64) return launch_cta<T, TR, 2>(p, num_sms, pdl, st);
        if (n <= 2048) return launch_cta<T, TR, 4>(p, num_sms, pdl, st);
        return launch_vec<T, TR, 8, false>(p, num_sms, (n + 255) / 256 * 32, pdl, st);
    }
    // single elements: 8 or 16 to a thread while a row fits 512 threads
    auto any = [&](auto kernel, int each, int most) {
        const int threads = std::min(most, ((p.H + each - 1) / each + 31) / 32 * 32);
        return launch_kernel(kernel, balanced(p.T, num_sms, threads), dim3(threads), 0, st, pdl, 1,
                             p);
    };
    if (p.H <= 8 * 512) return any(k_block_any<T, TR, 8>, 8, 512);
    if (p.H <= 16 * 512) return any(k_block_any<T, TR, 16>, 16, 512);
    return any(k_block_any<T, TR, 0>, 1, 1024);
}

}  // namespace block
}  // namespace rarn
