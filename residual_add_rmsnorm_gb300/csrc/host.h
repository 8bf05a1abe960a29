// host.h -- what the C ABI's translation units share on the host: the current
// device's properties, the launch setting and the error record of api.cu.
#pragma once

#include <cuda_runtime.h>

#include "../../include/rarn.h"

namespace rarn {
namespace host {

struct Device {
    int num_sms;
    int max_smem_optin;
    unsigned int *watchdog;  // the watchdog word's device address
};

// The current device; RARN_ERR_CUDA where there is none.
rarn_status current_device(Device *out);
// Records a CUDA error for rarn_last_cuda_error and returns RARN_ERR_CUDA.
rarn_status cuda_failed(cudaError_t e);
// The test hook's fill and limit (rarn_test_stall), once; false where none is set.
bool take_stall(long long *fill, unsigned long long *limit_ns);
// Whether launches carry the programmatic-serialization attribute.
bool pdl_enabled();

}  // namespace host
}  // namespace rarn
