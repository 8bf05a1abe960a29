// block_norm.cuh -- the norms after and before a block with its gate and the
// residual stream between them:
//
//   n = x * rsqrt(mean(x^2) + eps) * x_gamma          (x_gamma absent: n = x)
//   h = RN(residual_scale * r + scale * (gate * n))   the stream's type
//   y = RN(h * rsqrt(mean(h^2) + eps) * gamma)
//
// Two dependent sums over the row, binary32 throughout; h is normalised as it is
// stored.  Bound by memory: x and r are read, h and y written once.
#pragma once

#include "kv.cuh"

namespace rarn {
namespace block {

struct Params {
    const void *x, *residual;   // [T, H]
    void *h, *y;                // [T, H]; h may be residual, y may be x
    const void *gate;           // [gates, H] or nullptr
    const int32_t *index;       // [T]: the gate's row of each token, or nullptr
    const void *x_gamma, *gamma;  // [H]; x_gamma may be nullptr
    int64_t ldx, ldr, ldh, ldy, ldg;  // elements between rows; ldg 0: one row for all
    int64_t gates, T;
    int H;
    float eps, scale, residual_scale;
    unsigned int *watchdog;
};

// The gate's row of token t; -1 where the token's index lies outside the gate.
__device__ __forceinline__ int64_t gate_row(const Params &p, int64_t t) {
    if (!p.index) return p.gates == 1 ? 0 : t;
    const int64_t g = p.index[t];
    return g >= 0 && g < p.gates ? g : -1;
}

// Any row length, stride and alignment: a CTA per row, element by element, x and
// the new residual read again for the passes behind the sums (each thread what it
// read or wrote itself).
template <typename T, typename TR>
__global__ void __launch_bounds__(1024) k_block_any(const Params p) {
    __shared__ float red[2][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const float inv_h = 1.f / static_cast<float>(p.H);
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const T *x = static_cast<const T *>(p.x) + t * p.ldx;
        const TR *r = static_cast<const TR *>(p.residual) + t * p.ldr;
        TR *h = static_cast<TR *>(p.h) + t * p.ldh;
        T *y = static_cast<T *>(p.y) + t * p.ldy;
        const T *gate = nullptr;
        if (p.gate) {
            const int64_t g = gate_row(p, t);
            if (g < 0) {  // the whole CTA
                if (threadIdx.x == 0) atomicOr(p.watchdog, kv::kWatchIndex);
                continue;
            }
            gate = static_cast<const T *>(p.gate) + g * p.ldg;
        }
        float inv = 1.f;
        if (p.x_gamma) {
            float ss = 0.f;
            for (int i = threadIdx.x; i < p.H; i += blockDim.x) {
                const float v = DT<T>::to_f(x[i]);
                ss = fmaf(v, v, ss);
            }
            inv = rsqrtf(fmaf(block_sum(ss, red[0]), inv_h, p.eps));
        }
        float ss = 0.f;
        for (int i = threadIdx.x; i < p.H; i += blockDim.x) {
            float n = DT<T>::to_f(x[i]);
            if (p.x_gamma) n = n * inv * ld_elem<T>(p.x_gamma, i);
            if (gate) n *= DT<T>::to_f(gate[i]);
            const TR s =
                DT<TR>::from_f(fmaf(p.residual_scale, DT<TR>::to_f(r[i]), p.scale * n));
            h[i] = s;
            const float v = DT<TR>::to_f(s);
            ss = fmaf(v, v, ss);
        }
        const float inv2 = rsqrtf(fmaf(block_sum(ss, red[1]), inv_h, p.eps));
        for (int i = threadIdx.x; i < p.H; i += blockDim.x)
            y[i] = DT<T>::from_f(DT<TR>::to_f(h[i]) * inv2 * ld_elem<T>(p.gamma, i));
        __syncthreads();  // red is written again for the next row
    }
}

// Host launcher (instantiated per storage type; TR: the residual's).
template <typename T, typename TR>
cudaError_t launch_block(const Params &p, bool vec, int num_sms, bool pdl, cudaStream_t st);

}  // namespace block
}  // namespace rarn
