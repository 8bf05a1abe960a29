// tree_attn_launch.cuh -- host side of tree_attn.cuh: plan and launch.
#pragma once

#include <atomic>

#include "tree_attn.cuh"
#include "tree_plan.h"

namespace rarn {
namespace tree {

// CTAs of a kernel that the current device holds at once, asked for once per
// device.
template <typename K>
inline cudaError_t resident(K kernel, int threads, int num_sms, std::atomic<int> *known,
                            int *ctas) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<int> &slot = known[dev & 63];
    int per = slot.load(std::memory_order_relaxed);
    if (per == 0) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, 0);
        if (e != cudaSuccess) return e;
        if (per < 1) return cudaErrorInvalidConfiguration;
        slot.store(per, std::memory_order_relaxed);
    }
    *ctas = per * num_sms < kMaxCtas ? per * num_sms : kMaxCtas;
    return cudaSuccess;
}

template <int D, int NQ, bool kE5M2>
inline cudaError_t launch_rows(const Params &p, int num_sms, bool pdl, cudaStream_t st) {
    // loading a step ahead doubles the staging registers: only where the
    // accumulators leave room
    constexpr bool kAhead = NQ == 1 && D <= 128;
    static std::atomic<int> known[64];
    auto kernel = k_tree_rows<D, NQ, kE5M2, kAhead>;
    int ctas = 0;
    cudaError_t e = resident(kernel, kThreads, num_sms, known, &ctas);
    if (e != cudaSuccess) return e;
    if ((e = launch_kernel(kernel, dim3(ctas), dim3(kThreads), 0, st, pdl, 1, p)) != cudaSuccess)
        return e;
    return launch_kernel(k_tree_join<D>, dim3(p.max_segs, (8 * NQ + 7) / 8), dim3(256), 0, st,
                         pdl, 1, p, 8 * NQ, kTile);
}

template <int D, bool kE5M2>
inline cudaError_t launch_dim(const Params &p, const Plan &pl, int num_sms, bool pdl,
                              cudaStream_t st) {
    if constexpr (D <= 128)
        if (pl.rows == 16) return launch_rows<D, 2, kE5M2>(p, num_sms, pdl, st);
    return launch_rows<D, 1, kE5M2>(p, num_sms, pdl, st);
}

template <bool kE5M2>
cudaError_t launch_tree(const Params &p, const Plan &pl, int num_sms, bool pdl, cudaStream_t st) {
    switch (p.D) {
    case 64: return launch_dim<64, kE5M2>(p, pl, num_sms, pdl, st);
    case 96: return launch_dim<96, kE5M2>(p, pl, num_sms, pdl, st);
    case 128: return launch_dim<128, kE5M2>(p, pl, num_sms, pdl, st);
    case 192: return launch_dim<192, kE5M2>(p, pl, num_sms, pdl, st);
    default: return launch_dim<256, kE5M2>(p, pl, num_sms, pdl, st);
    }
}

}  // namespace tree
}  // namespace rarn
