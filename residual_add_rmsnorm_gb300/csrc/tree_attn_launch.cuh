// tree_attn_launch.cuh -- host side of tree_attn.cuh: plan and launch.
#pragma once

#include <atomic>

#include "gemm_norm_launch.cuh"  // tensor_map_encoder
#include "tree_attn.cuh"
#include "tree_plan.h"
#include "tree_tile.cuh"

namespace rarn {
namespace tree {

// CTAs of a kernel that the current device holds at once; the kernel's shared
// memory is allowed for and the question asked once per device.
template <typename K>
inline cudaError_t resident(K kernel, int threads, int smem, int num_sms, int most,
                            std::atomic<int> *known, int *ctas) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<int> &slot = known[dev & 63];
    int per = slot.load(std::memory_order_relaxed);
    if (per == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem);
        if (e != cudaSuccess) return e;
        if (per < 1) return cudaErrorInvalidConfiguration;
        slot.store(per, std::memory_order_relaxed);
    }
    *ctas = per * num_sms < most ? per * num_sms : most;
    return cudaSuccess;
}

// many: most segments are expected to have four parts or more.
template <int D>
inline cudaError_t launch_join(const Params &p, int rows, bool many, bool pdl, cudaStream_t st) {
    return many ? launch_kernel(k_tree_join<D, 8>, dim3(p.max_segs, rows), dim3(256), 0, st, pdl,
                                1, p, rows)
                : launch_kernel(k_tree_join<D, 1>, dim3(p.max_segs, (rows + 7) / 8), dim3(256), 0,
                                st, pdl, 1, p, rows);
}

// The codes of one tensor as a 4-D tensor [pages][heads][slots][D], boxes of
// `slots` slots by at most 128 bytes, stored in StepLayout's order.
template <int D>
inline bool encode_codes(CUtensorMap *map, const void *base, const Cache &c, int slots) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    using L = StepLayout<D>;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)c.page_size, (cuuint64_t)c.heads,
                                (cuuint64_t)c.pages};
    // the stride of a dimension of one is never used, but must be valid
    auto stride = [](int64_t s, int64_t n) { return (cuuint64_t)(n > 1 ? s : 16); };
    const cuuint64_t strides[3] = {stride(c.slot_stride, c.page_size),
                                   stride(c.head_stride, c.heads), stride(c.page_stride, c.pages)};
    const cuuint32_t box[4] = {(cuuint32_t)L::kHalf, (cuuint32_t)slots, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               L::kHalf == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NQ, int NP, bool kE5M2, bool kTma>
inline cudaError_t launch_rows(const Params &p, const Plan &pl, int num_sms, bool pdl,
                               cudaStream_t st) {
    // what a warp keeps in flight: about 8 KB of keys and values behind the
    // step that it works on
    constexpr int kStages = D >= 128 ? 3 : 4;
    using S = Smem<D, NQ, kStages>;
    static std::atomic<int> known[64];
    auto kernel = k_tree_rows<D, NQ, NP, kE5M2, kStages, kTma>;
    CUtensorMap km{}, vm{};
    if (kTma && !(encode_codes<D>(&km, p.cache.k, p.cache, kStep) &&
                  encode_codes<D>(&vm, p.cache.v, p.cache, kStep)))
        return cudaErrorInvalidValue;
    int ctas = 0;
    cudaError_t e = resident(kernel, kThreads, S::kBytes, num_sms, kMaxCtas, known, &ctas);
    if (e != cudaSuccess) return e;
    if ((e = launch_kernel(kernel, dim3(ctas), dim3(kThreads), S::kBytes, st, pdl, 1, p, km,
                           vm)) != cudaSuccess)
        return e;
    return launch_join<D>(p, 8 * NQ, ctas >= 4 * pl.expected, pdl, st);
}

template <int D, int NP, bool kE5M2, bool kTma>
inline cudaError_t launch_dim(const Params &p, const Plan &pl, int num_sms, bool pdl,
                              cudaStream_t st) {
    if constexpr (D <= 192)
        if (pl.rows == 16) return launch_rows<D, 2, NP, kE5M2, kTma>(p, pl, num_sms, pdl, st);
    return launch_rows<D, 1, NP, kE5M2, kTma>(p, pl, num_sms, pdl, st);
}

template <int D, bool kE5M2, bool kTma>
inline cudaError_t launch_copies(const Params &p, const Plan &pl, int num_sms, bool pdl,
                                 cudaStream_t st) {
    return p.bf16 ? launch_dim<D, 2, kE5M2, kTma>(p, pl, num_sms, pdl, st)
                  : launch_dim<D, 3, kE5M2, kTma>(p, pl, num_sms, pdl, st);
}

// TMA boxes need steps inside a page and adjacent scales (Params::whole_steps).
template <int D, bool kE5M2>
inline cudaError_t launch_type(const Params &p, const Plan &pl, int num_sms, bool pdl,
                               cudaStream_t st) {
    if constexpr (rows_by_tma(D))
        if (p.whole_steps) return launch_copies<D, kE5M2, true>(p, pl, num_sms, pdl, st);
    return launch_copies<D, kE5M2, false>(p, pl, num_sms, pdl, st);
}

template <int D, int NP, bool kE5M2, bool kTwo>
inline cudaError_t launch_tiles(const Params &given, const Plan &pl, int num_sms, bool pdl,
                                cudaStream_t st) {
    static std::atomic<int> known[64];
    auto kernel = k_tree_tile<D, NP, kE5M2, kTwo>;
    constexpr int smem = TileSmem<D, NP, kTwo>::kBytes;
    CUtensorMap km{}, vm{};
    // The largest boxes that lie inside a page and a tile.
    Params p = given;
    for (p.box = kBox; p.box < kTileKeys && p.cache.page_size % (2 * p.box) == 0;) p.box *= 2;
    if (!encode_codes<D>(&km, p.cache.k, p.cache, p.box) ||
        !encode_codes<D>(&vm, p.cache.v, p.cache, p.box))
        return cudaErrorInvalidValue;
    int ctas = 0;
    cudaError_t e = resident(kernel, kTileThreads, smem, num_sms, kMaxTileCtas, known, &ctas);
    if (e != cudaSuccess) return e;
    if ((e = launch_kernel(kernel, dim3(ctas), dim3(kTileThreads), smem, st, pdl, 1, p, km, vm)) !=
        cudaSuccess)
        return e;
    return launch_join<D>(p, pl.rows, ctas >= 4 * pl.expected, pdl, st);
}

template <int D, bool kE5M2>
inline cudaError_t launch_tile_type(const Params &p, const Plan &pl, int num_sms, bool pdl,
                                    cudaStream_t st) {
    if (pl.rows == 256)
        return p.bf16 ? launch_tiles<D, 2, kE5M2, true>(p, pl, num_sms, pdl, st)
                      : launch_tiles<D, 3, kE5M2, true>(p, pl, num_sms, pdl, st);
    return p.bf16 ? launch_tiles<D, 2, kE5M2, false>(p, pl, num_sms, pdl, st)
                  : launch_tiles<D, 3, kE5M2, false>(p, pl, num_sms, pdl, st);
}

template <bool kE5M2>
cudaError_t launch_tree(const Params &p, const Plan &pl, int num_sms, bool pdl, cudaStream_t st) {
    if (pl.tiles)
        return p.D == 64 ? launch_tile_type<64, kE5M2>(p, pl, num_sms, pdl, st)
                         : launch_tile_type<128, kE5M2>(p, pl, num_sms, pdl, st);
    switch (p.D) {
    case 64: return launch_type<64, kE5M2>(p, pl, num_sms, pdl, st);
    case 96: return launch_type<96, kE5M2>(p, pl, num_sms, pdl, st);
    case 128: return launch_type<128, kE5M2>(p, pl, num_sms, pdl, st);
    case 192: return launch_type<192, kE5M2>(p, pl, num_sms, pdl, st);
    default: return launch_type<256, kE5M2>(p, pl, num_sms, pdl, st);
    }
}

}  // namespace tree
}  // namespace rarn
