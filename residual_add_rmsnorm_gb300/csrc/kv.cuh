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

// Four codes to two pairs of binary16, exactly (both formats are subsets of
// it).  One instruction per pair; the header's intrinsic, which returns the
// halves apart, measured three times that.
template <bool kE5M2>
__device__ __forceinline__ void codes4_to_h2(uint32_t four, uint32_t &lo, uint32_t &hi) {
    if constexpr (kE5M2) {
        asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\n"
            "cvt.rn.f16x2.e5m2x2 %0, a;\ncvt.rn.f16x2.e5m2x2 %1, b;\n}\n"
            : "=r"(lo), "=r"(hi)
            : "r"(four));
    } else {
        asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\n"
            "cvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
            : "=r"(lo), "=r"(hi)
            : "r"(four));
    }
}

template <bool kE5M2>
__device__ __forceinline__ uint32_t codes2_to_h2(uint32_t two) {
    uint32_t lo, hi;
    codes4_to_h2<kE5M2>(two, lo, hi);
    return lo;
}

__device__ __forceinline__ float2 codes2_to_f2(uint32_t two, int fmt) {
    const uint32_t h = fmt == Q_E5M2 ? codes2_to_h2<true>(two) : codes2_to_h2<false>(two);
    return DT<__half>::w2f(h);
}

}  // namespace kv
}  // namespace rarn
