// verify_launch.cuh -- host side of verify.cuh: how many CTAs take a sequence.
#pragma once

#include "verify.cuh"

#ifndef VF_CAP
#define VF_CAP 4
#endif
namespace rarn {
namespace verify {

template <typename T>
cudaError_t launch_verify(const Params &p, int num_sms, bool pdl, cudaStream_t st) {
    int cluster = kMaxCluster;
    while (cluster > 1 && (int64_t)p.B * cluster > VF_CAP * num_sms) cluster /= 2;
    return launch_kernel(k_verify<T>, dim3((unsigned)(p.B * cluster)), dim3(kThreads), 0, st, pdl,
                         cluster, p, cluster);
}

}  // namespace verify
}  // namespace rarn
