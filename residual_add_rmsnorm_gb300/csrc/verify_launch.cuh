// verify_launch.cuh -- host side of verify.cuh: how many CTAs take a sequence.
#pragma once

#include "verify.cuh"

namespace rarn {
namespace verify {

template <typename T>
cudaError_t launch_verify(const Params &p, int num_sms, bool pdl, cudaStream_t st) {
    // as many as the SMs hold at once, four each (64 sequences, 128256 tokens of p and q
    // in binary32: 13.5 us; at most two or three each 14.4, eight 13.6; 256 sequences, 32000
    // tokens in bfloat16: 10.5, 10.1, 14.0)
    int cluster = kMaxCluster;
    while (cluster > 1 && (int64_t)p.B * cluster > 4 * num_sms) cluster /= 2;
    return launch_kernel(k_verify<T>, dim3((unsigned)(p.B * cluster)), dim3(kThreads), 0, st, pdl,
                         cluster, p, cluster);
}

}  // namespace verify
}  // namespace rarn
