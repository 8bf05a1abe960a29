// block_api.cu -- the C ABI of the norms around a block (rarn_gated_add_rms_norm):
// argument checks before anything is enqueued, one launch, no memory allocated.
#include <cmath>

#include "../../include/rarn.h"
#include "block_norm.cuh"
#include "host.h"
#include "kv_check.h"

namespace rarn {
namespace block {
// instantiated in block_norm_{bf16,f16,f32}.cu
extern template cudaError_t launch_block<__nv_bfloat16, __nv_bfloat16>(const Params &, bool, int,
                                                                       bool, cudaStream_t);
extern template cudaError_t launch_block<__nv_bfloat16, float>(const Params &, bool, int, bool,
                                                               cudaStream_t);
extern template cudaError_t launch_block<__half, __half>(const Params &, bool, int, bool,
                                                         cudaStream_t);
extern template cudaError_t launch_block<__half, float>(const Params &, bool, int, bool,
                                                        cudaStream_t);
extern template cudaError_t launch_block<float, float>(const Params &, bool, int, bool,
                                                       cudaStream_t);
}  // namespace block
}  // namespace rarn

using namespace rarn;
using namespace rarn::check;

namespace {

rarn_status check_rows(const rarn_rows &m, int64_t T, int64_t H) {
    if (!m.data || m.row_stride < 0 || (T > 1 && m.row_stride < H)) return RARN_ERR_INVALID_ARG;
    if (!reaches(m.row_stride, T)) return RARN_ERR_UNSUPPORTED;
    return on(m.data, (unsigned)size_of(m.dtype)) ? RARN_OK : RARN_ERR_INVALID_ARG;
}

Range span_of(const rarn_rows &m, int64_t T, int64_t H) {
    return solid(m.data, ((T - 1) * (T > 1 ? m.row_stride : 0) + H) * size_of(m.dtype));
}

bool same(const rarn_rows &a, const rarn_rows &b, int64_t T) {
    return a.data == b.data && a.dtype == b.dtype && (T == 1 || a.row_stride == b.row_stride);
}

bool packs_ok(const rarn_rows &m, int64_t T) {
    return on(m.data, 16) && (T == 1 || m.row_stride * size_of(m.dtype) % 16 == 0);
}

}  // namespace

extern "C" rarn_status rarn_gated_add_rms_norm(rarn_rows y, rarn_rows residual_out, rarn_rows x,
                                               rarn_rows residual, const void *x_gamma,
                                               const void *gamma, const rarn_gate *gate,
                                               float scale, float residual_scale, int64_t T,
                                               int64_t H, float eps, void *stream) {
    if (!type_ok(x.dtype) || !type_ok(y.dtype) || !type_ok(residual.dtype) ||
        !type_ok(residual_out.dtype))
        return RARN_ERR_INVALID_ARG;
    if (T < 0 || H <= 0 || !(eps >= 0.f) || std::isinf(eps) || !std::isfinite(scale) ||
        !std::isfinite(residual_scale))
        return RARN_ERR_INVALID_ARG;
    if (H > RARN_MAX_H || T > RARN_MAX_T) return RARN_ERR_UNSUPPORTED;
    if (gate && gate->rows < 0) return RARN_ERR_INVALID_ARG;
    // without tokens a gate for each has no rows, and their indices no address
    if (gate && T > 0 &&
        (gate->rows < 1 || (!gate->index && gate->rows != 1 && gate->rows != T)))
        return RARN_ERR_INVALID_ARG;
    if (y.dtype != x.dtype || residual_out.dtype != residual.dtype ||
        (residual.dtype != x.dtype && residual.dtype != RARN_F32))
        return RARN_ERR_UNSUPPORTED;
    if (T == 0) return RARN_OK;
    rarn_status st;
    for (const rarn_rows *m : {&y, &residual_out, &x, &residual})
        if ((st = check_rows(*m, T, H)) != RARN_OK) return st;
    const int64_t s = size_of(x.dtype);
    if (!gamma || !on(gamma, (unsigned)s) || !on(x_gamma, (unsigned)s)) return RARN_ERR_INVALID_ARG;
    rarn_rows g{};
    if (gate) {
        g = rarn_rows{const_cast<void *>(gate->data), gate->row_stride, x.dtype};
        if ((st = check_rows(g, gate->rows, H)) != RARN_OK) return st;
        if (!on(gate->index, 4)) return RARN_ERR_INVALID_ARG;
    }
    // y may be x and residual_out the residual, exactly; nothing else may meet
    const Range yr = span_of(y, T, H), hr = span_of(residual_out, T, H);
    const Range xr = span_of(x, T, H), rr = span_of(residual, T, H);
    if (meet(yr, hr) || (!same(y, x, T) && meet(yr, xr)) || meet(yr, rr) || meet(hr, xr) ||
        (!same(residual_out, residual, T) && meet(hr, rr)))
        return RARN_ERR_ALIAS;
    for (const Range &o : {yr, hr}) {
        if (meet(o, solid(gamma, H * s)) || (x_gamma && meet(o, solid(x_gamma, H * s))))
            return RARN_ERR_ALIAS;
        if (gate && (meet(o, span_of(g, gate->rows, H)) ||
                     (gate->index && meet(o, solid(gate->index, T * 4)))))
            return RARN_ERR_ALIAS;
    }
    host::Device dev;
    if ((st = host::current_device(&dev)) != RARN_OK) return st;
    block::Params p{};
    p.x = x.data;
    p.residual = residual.data;
    p.h = residual_out.data;
    p.y = y.data;
    p.x_gamma = x_gamma;
    p.gamma = gamma;
    p.ldx = x.row_stride;
    p.ldr = residual.row_stride;
    p.ldh = residual_out.row_stride;
    p.ldy = y.row_stride;
    if (gate) {
        p.gate = gate->data;
        p.index = gate->index;
        p.gates = gate->rows;
        p.ldg = gate->rows > 1 ? gate->row_stride : 0;
    }
    p.T = T;
    p.H = (int)H;
    p.eps = eps;
    p.scale = scale;
    p.residual_scale = residual_scale;
    p.watchdog = dev.watchdog;
    const bool vec = H * s % 16 == 0 && packs_ok(y, T) && packs_ok(x, T) && packs_ok(residual, T) &&
                     packs_ok(residual_out, T) && on(gamma, 16) && on(x_gamma, 16) &&
                     (!gate || packs_ok(g, gate->rows));
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool pdl = host::pdl_enabled();
    const bool wide = residual.dtype == RARN_F32;
    cudaError_t e;
    switch (x.dtype) {
    case RARN_BF16:
        e = wide ? block::launch_block<__nv_bfloat16, float>(p, vec, dev.num_sms, pdl, cs)
                 : block::launch_block<__nv_bfloat16, __nv_bfloat16>(p, vec, dev.num_sms, pdl, cs);
        break;
    case RARN_F16:
        e = wide ? block::launch_block<__half, float>(p, vec, dev.num_sms, pdl, cs)
                 : block::launch_block<__half, __half>(p, vec, dev.num_sms, pdl, cs);
        break;
    default: e = block::launch_block<float, float>(p, vec, dev.num_sms, pdl, cs); break;
    }
    return e == cudaSuccess ? RARN_OK : host::cuda_failed(e);
}
