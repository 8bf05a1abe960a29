// kv.cuh -- views of the attention-side kernels: [T, heads, D] matrices inside
// larger allocations, and the paged 8-bit key / value cache.
#pragma once

#include "common.cuh"

namespace rarn {
namespace kv {

// Watchdog bit: an index in device memory (a position, a cache slot, a page)
// lay outside its table; what it named was left out.
constexpr unsigned int kWatchIndex = 16u;

// [T, heads, D] with unit stride inside a head; strides in elements.
struct Heads {
    void *data;
    int64_t ts, hs;
    int heads;
};

// Keys and values as one-byte codes with binary32 scales.  Code strides in
// bytes, scale strides in elements; the same for keys and values.
struct Cache {
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    int64_t page_stride, head_stride, slot_stride;
    int64_t s_page, s_head, s_slot;  // zero with one scale per tensor
    int64_t pages;
    int page_size;
    int heads;
    int fmt;   // QFormat
    int mode;  // QMode
};

// Two codes to binary16, exactly (both formats are subsets of it).
template <bool kE5M2>
__device__ __forceinline__ uint32_t codes2_to_h2(uint32_t two) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two),
                                                     kE5M2 ? __NV_E5M2 : __NV_E4M3);
    return static_cast<uint32_t>(r.x) | (static_cast<uint32_t>(r.y) << 16);
}

__device__ __forceinline__ float2 codes2_to_f2(uint32_t two, int fmt) {
    const uint32_t h = fmt == Q_E5M2 ? codes2_to_h2<true>(two) : codes2_to_h2<false>(two);
    return DT<__half>::w2f(h);
}

}  // namespace kv
}  // namespace rarn
