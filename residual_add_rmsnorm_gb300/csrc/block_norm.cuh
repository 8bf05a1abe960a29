// block_norm.cuh -- the norms after and before a block with its gate and the
// residual stream between them:
//
//   n = x * rsqrt(mean(x^2) + eps) * x_gamma          (x_gamma absent: n = x)
//   h = RN(residual_scale * r + scale * (gate * n))   the stream's type
//   y = RN(h * rsqrt(mean(h^2) + eps) * gamma)
//
// Two dependent sums over the row, binary32 throughout; h is normalised as it is
// stored.  Bound by memory: x and r are read, h and y written once, the row stays in
// registers between the sums.  Measured, bfloat16: 16384 rows of 5120 with one gate
// 107 us (92 % of a copy's rate; without a gate 96), 8192 of 8192 81 us (97 %), 517 of
// 5120 with a binary32 residual and gates 7.1 us (66 %: one wave that reads, sums twice
// and writes), one row of 4096 1.9 us.  What a gated row lacks is its instructions:
// conversions from 16 bits are half of the 25 an element takes, and issue slots are half
// full.
#pragma once

#include "kv.cuh"
#include "rows.cuh"

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

// Rows in registers, 16-byte packs: a CTA of n / 4 threads per row, down to one warp.
// Between the sums a thread keeps its packs of x and r as they came and then of h as
// it is stored, so that nothing is read twice; the gammas and shared gates come from
// L1.  kPipe: the next row's loads are under way while a row is summed and written.
template <typename T, typename TR, int VPT>
struct RowPacks {
    uint4 x[VPT], r[VPT][Res<T, TR>::N];
};

template <typename T, typename TR, int VPT, bool kFull>
__device__ __forceinline__ void load_row(const Params &p, int64_t t, int j0, int js, int nv,
                                         RowPacks<T, TR, VPT> &b) {
    using RS = Res<T, TR>;
    const T *x = static_cast<const T *>(p.x) + t * p.ldx;
    const TR *r = static_cast<const TR *>(p.residual) + t * p.ldr;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int j = j0 + k * js;
        if (kFull || j < nv) {
            b.x[k] = ld_stream(x + j * RS::EPV);
#pragma unroll
            for (int q = 0; q < RS::N; ++q)
                b.r[k][q] = ld_stream(r + j * RS::EPV + q * RS::EPW);
        }
    }
}

// Threads that a CTA of the kernel may have and CTAs to an SM, which set its registers.
// Four packs a thread and the next row's take 128, and fewer cost more than the warps
// that they would leave room for (16384 rows of 5120, binary32 residual: 155 us with
// 128, 195 with 102, 250 with 85); a row alone leaves room for four CTAs of 160.
template <int VPT, bool kPipe, bool kFull>
constexpr int kMaxThreads = VPT == 1 ? 1024 : VPT == 4 && !kPipe && kFull ? 320 : 512;
template <int VPT, bool kPipe, bool kFull>
constexpr int kMinCtas = VPT == 4 && !kPipe && kFull ? 2 : 1;

// Packs as pairs, for arithmetic two elements to an instruction.
template <typename T>
__device__ __forceinline__ void unpack2(const uint4 &p, float2 (&f)[DT<T>::EPV / 2]) {
    if constexpr (sizeof(T) == 4) {
        f[0] = float2{__uint_as_float(p.x), __uint_as_float(p.y)};
        f[1] = float2{__uint_as_float(p.z), __uint_as_float(p.w)};
    } else {
        f[0] = DT<T>::w2f(p.x);
        f[1] = DT<T>::w2f(p.y);
        f[2] = DT<T>::w2f(p.z);
        f[3] = DT<T>::w2f(p.w);
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack2(const float2 (&f)[DT<T>::EPV / 2]) {
    if constexpr (sizeof(T) == 4)
        return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y),
                          __float_as_uint(f[1].x), __float_as_uint(f[1].y));
    else
        return make_uint4(DT<T>::f2w(f[0].x, f[0].y), DT<T>::f2w(f[1].x, f[1].y),
                          DT<T>::f2w(f[2].x, f[2].y), DT<T>::f2w(f[3].x, f[3].y));
}

// The residual's words of one pack of T.
template <typename T, typename TR>
__device__ __forceinline__ void res_unpack2(const uint4 (&v)[Res<T, TR>::N],
                                            float2 (&f)[DT<T>::EPV / 2]) {
    if constexpr (Res<T, TR>::SAME) {
        unpack2<T>(v[0], f);
    } else {
#pragma unroll
        for (int q = 0; q < Res<T, TR>::N; ++q) {
            f[2 * q] = float2{__uint_as_float(v[q].x), __uint_as_float(v[q].y)};
            f[2 * q + 1] = float2{__uint_as_float(v[q].z), __uint_as_float(v[q].w)};
        }
    }
}

template <typename T, typename TR>
__device__ __forceinline__ void res_pack2(const float2 (&f)[DT<T>::EPV / 2],
                                          uint4 (&v)[Res<T, TR>::N]) {
    if constexpr (Res<T, TR>::SAME) {
        v[0] = pack2<T>(f);
    } else {
#pragma unroll
        for (int q = 0; q < Res<T, TR>::N; ++q)
            v[q] = make_uint4(__float_as_uint(f[2 * q].x), __float_as_uint(f[2 * q].y),
                              __float_as_uint(f[2 * q + 1].x), __float_as_uint(f[2 * q + 1].y));
    }
}

// kFull: every thread has VPT packs, none is checked against the row's end.
template <typename T, typename TR, int VPT, bool kGate, bool kPipe, bool kFull>
__global__ void __launch_bounds__(kMaxThreads<VPT, kPipe, kFull>, kMinCtas<VPT, kPipe, kFull>)
    k_block_vec(const Params p) {
    using RS = Res<T, TR>;
    constexpr int E = RS::EPV;
    __shared__ float red[4][32];
    const int nv = p.H / E, j0 = threadIdx.x, js = blockDim.x;
    const int64_t step = gridDim.x;
    int64_t t = blockIdx.x;
    const float inv_h = 1.f / static_cast<float>(p.H);
    const T *xg = static_cast<const T *>(p.x_gamma), *gm = static_cast<const T *>(p.gamma);
    grid_dependency_wait();
    grid_launch_dependents();
    // two sums a row, each in a buffer that the row before did not use
    int par = 0;
    auto row_sum = [&](float v, int which) { return block_sum(v, red[2 * par + which]); };
    RowPacks<T, TR, VPT> next;
    if (kPipe && t < p.T) load_row<T, TR, VPT, kFull>(p, t, j0, js, nv, next);
    for (; t < p.T; t += step, par ^= 1) {
        RowPacks<T, TR, VPT> cur;
        if constexpr (kPipe) cur = next;
        else load_row<T, TR, VPT, kFull>(p, t, j0, js, nv, cur);
        uint4 gate[kGate ? VPT : 1];
        bool live = true;
        if constexpr (kGate) {
            const int64_t g = gate_row(p, t);
            live = g >= 0;  // else the row is only gone through
            const T *row = static_cast<const T *>(p.gate) + (live ? g : 0) * p.ldg;
            if (!live && j0 == 0) atomicOr(p.watchdog, kv::kWatchIndex);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int j = j0 + k * js;
                if (kFull || j < nv) gate[k] = ld_stream(row + j * E);
            }
        }
        if constexpr (kPipe)
            if (t + step < p.T) load_row<T, TR, VPT, kFull>(p, t + step, j0, js, nv, next);
        if constexpr (!kPipe) {  // the next row into L2 (2000 rows of 16384: 133 -> 126 us)
            if (j0 == 0 && t + step < p.T) {
                prefetch_l2(static_cast<const T *>(p.x) + (t + step) * p.ldx,
                            (uint32_t)(p.H * sizeof(T)));
                prefetch_l2(static_cast<const TR *>(p.residual) + (t + step) * p.ldr,
                            (uint32_t)(p.H * sizeof(TR)));
            }
        }
        float inv = 1.f;
        if (xg) {
            float2 ss = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if (kFull || j0 + k * js < nv) {
                    float2 x[E / 2];
                    unpack2<T>(cur.x[k], x);
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) ss = __ffma2_rn(x[e], x[e], ss);
                }
            }
            inv = rsqrtf(fmaf(row_sum(ss.x + ss.y, 0), inv_h, p.eps));
        }
        TR *h = static_cast<TR *>(p.h) + t * p.ldh;
        const float2 by = {inv, inv}, scale = {p.scale, p.scale};
        const float2 keep = {p.residual_scale, p.residual_scale};
        float2 ss = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int j = j0 + k * js;
            if (kFull || j < nv) {
                float2 n[E / 2], w[E / 2], s[E / 2];
                unpack2<T>(cur.x[k], n);
#pragma unroll
                for (int e = 0; e < E / 2; ++e) n[e] = __fmul2_rn(n[e], by);
                if (xg) {
                    unpack2<T>(ld_keep(xg + j * E), w);
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) n[e] = __fmul2_rn(n[e], w[e]);
                }
                if constexpr (kGate) {
                    unpack2<T>(gate[k], w);
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) n[e] = __fmul2_rn(n[e], w[e]);
                }
                res_unpack2<T, TR>(cur.r[k], s);
#pragma unroll
                for (int e = 0; e < E / 2; ++e)
                    s[e] = __ffma2_rn(keep, s[e], __fmul2_rn(scale, n[e]));
                res_pack2<T, TR>(s, cur.r[k]);
                if (live) {
#pragma unroll
                    for (int q = 0; q < RS::N; ++q)
                        st_global(h + j * E + q * RS::EPW, cur.r[k][q]);
                }
                res_unpack2<T, TR>(cur.r[k], s);
#pragma unroll
                for (int e = 0; e < E / 2; ++e) ss = __ffma2_rn(s[e], s[e], ss);
            }
        }
        const float inv2 = rsqrtf(fmaf(row_sum(ss.x + ss.y, 1), inv_h, p.eps));
        T *y = static_cast<T *>(p.y) + t * p.ldy;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int j = j0 + k * js;
            if (kFull || j < nv) {
                float2 s[E / 2], w[E / 2];
                res_unpack2<T, TR>(cur.r[k], s);
                unpack2<T>(ld_keep(gm + j * E), w);
#pragma unroll
                for (int e = 0; e < E / 2; ++e)
                    s[e] = __fmul2_rn(__fmul2_rn(s[e], float2{inv2, inv2}), w[e]);
                if (live) st_global(y + j * E, pack2<T>(s));
            }
        }
    }
}

// An element of a gamma, which no output overlaps: a load that stores do not hold back
// (a gate may come from the kernel just before: plain loads).
template <typename T>
__device__ __forceinline__ float ld_const(const void *base, int i) {
    if constexpr (sizeof(T) == 4) {
        return __ldg(static_cast<const float *>(base) + i);
    } else {
        const unsigned short w = __ldg(static_cast<const unsigned short *>(base) + i);
        return DT<T>::to_f(*reinterpret_cast<const T *>(&w));
    }
}

// Any row length, stride and alignment: a CTA per row, element by element.  With NE > 0
// a thread holds its NE elements from the first load on; NE == 0, rows longer than
// that: x and the new residual are read again for the passes behind the sums (each
// thread what it read or wrote itself).
template <typename T, typename TR, int NE>
__global__ void __launch_bounds__(NE > 0 ? 512 : 1024, NE > 0 ? 2 : 1)
    k_block_any(const Params p) {
    __shared__ float red[2][2][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const float inv_h = 1.f / static_cast<float>(p.H);
    const int js = blockDim.x, j0 = threadIdx.x;
    int par = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, par ^= 1) {
        const T *x = static_cast<const T *>(p.x) + t * p.ldx;
        const TR *r = static_cast<const TR *>(p.residual) + t * p.ldr;
        TR *h = static_cast<TR *>(p.h) + t * p.ldh;
        T *y = static_cast<T *>(p.y) + t * p.ldy;
        const T *gate = nullptr;
        bool live = true;
        if (p.gate) {
            const int64_t g = gate_row(p, t);
            live = g >= 0;
            gate = static_cast<const T *>(p.gate) + (live ? g : 0) * p.ldg;
            if (!live && j0 == 0) atomicOr(p.watchdog, kv::kWatchIndex);
        }
        float ss = 0.f, inv = 1.f;
        if constexpr (NE > 0) {
            // this thread's elements j0 + k * js; beyond the row its first one is read in
            // their place (of a thread that has none the row's first gamma) and weighs nothing
            int at[NE];
            float n[NE], s[NE], w[NE];
#pragma unroll
            for (int k = 0; k < NE; ++k)
                at[k] = j0 + k * js < p.H ? j0 + k * js : j0 < p.H ? j0 : 0;
#pragma unroll
            for (int k = 0; k < NE; ++k) n[k] = s[k] = 0.f;
            if (j0 < p.H) {
#pragma unroll
                for (int k = 0; k < NE; ++k) n[k] = DT<T>::to_f(x[at[k]]);
#pragma unroll
                for (int k = 0; k < NE; ++k) s[k] = DT<TR>::to_f(r[at[k]]);
            }
            if (p.x_gamma) {
#pragma unroll
                for (int k = 0; k < NE; ++k) w[k] = ld_const<T>(p.x_gamma, at[k]);
#pragma unroll
                for (int k = 0; k < NE; ++k) ss += j0 + k * js < p.H ? n[k] * n[k] : 0.f;
                inv = rsqrtf(fmaf(block_sum(ss, red[par][0]), inv_h, p.eps));
#pragma unroll
                for (int k = 0; k < NE; ++k) n[k] = n[k] * inv * w[k];
            }
            if (gate) {
#pragma unroll
                for (int k = 0; k < NE; ++k) w[k] = DT<T>::to_f(gate[at[k]]);
#pragma unroll
                for (int k = 0; k < NE; ++k) n[k] *= w[k];
            }
#pragma unroll
            for (int k = 0; k < NE; ++k) w[k] = ld_const<T>(p.gamma, at[k]);
            ss = 0.f;
#pragma unroll
            for (int k = 0; k < NE; ++k) {
                s[k] = DT<TR>::round(fmaf(p.residual_scale, s[k], p.scale * n[k]));
                ss += j0 + k * js < p.H ? s[k] * s[k] : 0.f;
            }
            const int end = live ? p.H : 0;
#pragma unroll
            for (int k = 0; k < NE; ++k)
                if (j0 + k * js < end) h[at[k]] = DT<TR>::from_f(s[k]);
            const float inv2 = rsqrtf(fmaf(block_sum(ss, red[par][1]), inv_h, p.eps));
#pragma unroll
            for (int k = 0; k < NE; ++k)
                if (j0 + k * js < end) y[at[k]] = DT<T>::from_f(s[k] * inv2 * w[k]);
        } else {
            if (p.x_gamma) {
                for (int i = j0; i < p.H; i += js) {
                    const float v = DT<T>::to_f(x[i]);
                    ss = fmaf(v, v, ss);
                }
                inv = rsqrtf(fmaf(block_sum(ss, red[par][0]), inv_h, p.eps));
            }
            ss = 0.f;
            for (int i = j0; i < p.H; i += js) {
                float v = DT<T>::to_f(x[i]);
                if (p.x_gamma) v = v * inv * ld_const<T>(p.x_gamma, i);
                if (gate) v *= DT<T>::to_f(gate[i]);
                v = DT<TR>::round(fmaf(p.residual_scale, DT<TR>::to_f(r[i]), p.scale * v));
                if (live) h[i] = DT<TR>::from_f(v);
                ss = fmaf(v, v, ss);
            }
            const float inv2 = rsqrtf(fmaf(block_sum(ss, red[par][1]), inv_h, p.eps));
            if (!live) continue;  // the whole CTA
            for (int i = j0; i < p.H; i += js)
                y[i] = DT<T>::from_f(DT<TR>::to_f(h[i]) * inv2 * ld_const<T>(p.gamma, i));
        }
    }
}

// Host launcher (instantiated per storage type; TR: the residual's).
template <typename T, typename TR>
cudaError_t launch_block(const Params &p, bool vec, int num_sms, bool pdl, cudaStream_t st);

}  // namespace block
}  // namespace rarn
