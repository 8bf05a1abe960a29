// kv_rows_launch.cuh -- host side of kv_rows.cuh: which kernel a call gets.
#pragma once

#include "kv_rows.cuh"

namespace rarn {
namespace kv {

// Heads per group at most, and warps per SM below which a call's heads are
// spread over more warps (8192 tokens of 64 + 8 heads: 57.9 us with 8 heads,
// 62.6 with 4, 61 with 16; 517 tokens of 40 + 8: 8.3 us with 16 warps, 10.3
// with 32 or 64, which leave a warp two loads).
constexpr int kRowHeads = 8;
constexpr int kRowWarps = 16;

template <typename T, int LG, bool kInter>
inline cudaError_t launch_head_group(const RowParams &p, int num_sms, bool pdl, cudaStream_t st) {
    constexpr int gpw = 32 / LG;
    auto chunks_of = [](int heads, int per) { return (heads + per * gpw - 1) / (per * gpw); };
    // Heads per group: as many as leave every SM its warps; the table's
    // products are formed once per warp.
    int per = kRowHeads;
    int nq, nk, nv;
    for (;; per /= 2) {
        nq = chunks_of(p.q.heads, per);
        nk = chunks_of(p.k.heads, per);
        nv = chunks_of(p.v.heads, per);
        if (per == 1 || p.T * (nq + nk + nv) >= (int64_t)num_sms * kRowWarps) break;
    }
    const int chunks = nq + nk + nv;
    return launch_kernel(k_head_rows<T, LG, kInter>, dim3((unsigned)((p.T + 3) / 4 * chunks)),
                         dim3(128), 0, st, pdl, 1, p, per, nq, nk, chunks);
}

template <typename T, int LG>
inline cudaError_t launch_head_style(const RowParams &p, int num_sms, bool pdl, cudaStream_t st) {
    return p.interleaved ? launch_head_group<T, LG, true>(p, num_sms, pdl, st)
                         : launch_head_group<T, LG, false>(p, num_sms, pdl, st);
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
    if (lanes <= 4) return launch_head_style<T, 4>(p, num_sms, pdl, st);
    if (lanes <= 8) return launch_head_style<T, 8>(p, num_sms, pdl, st);
    if (lanes <= 16) return launch_head_style<T, 16>(p, num_sms, pdl, st);
    return launch_head_style<T, 32>(p, num_sms, pdl, st);
}

template <typename T, int kStore, int kRows>
inline cudaError_t launch_read_rows(const ReadParams &p, bool pdl, cudaStream_t st) {
    const dim3 grid((unsigned)((p.rows + kRows - 1) / kRows));
    return p.cache.fmt == Q_E5M2 ? launch_kernel(k_cache_read<T, kStore, true, kRows>, grid,
                                                 dim3(kReadThreads), 0, st, pdl, 1, p)
                                 : launch_kernel(k_cache_read<T, kStore, false, kRows>, grid,
                                                 dim3(kReadThreads), 0, st, pdl, 1, p);
}

// 16 rows per CTA, or 8 while that leaves SMs without their four CTAs (2094
// rows 7.0 -> 6.4 us; 33 thousand rows 67.9 with 16, 72.0 with 8).
template <typename T, int kStore>
inline cudaError_t launch_read_format(const ReadParams &p, int num_sms, bool pdl,
                                      cudaStream_t st) {
    return p.rows < (int64_t)num_sms * 64 ? launch_read_rows<T, kStore, 8>(p, pdl, st)
                                          : launch_read_rows<T, kStore, 16>(p, pdl, st);
}

template <typename T>
cudaError_t launch_cache_read(const ReadParams &p, int store, int num_sms, bool pdl,
                              cudaStream_t st) {
    return store == 32   ? launch_read_format<T, 32>(p, num_sms, pdl, st)
           : store == 16 ? launch_read_format<T, 16>(p, num_sms, pdl, st)
                         : launch_read_format<T, 0>(p, num_sms, pdl, st);
}

}  // namespace kv
}  // namespace rarn
