// kv_check.h -- argument checks that the attention side's and the step's entry
// points share: types, strides, byte ranges that may not meet, the cache's
// descriptor, page tables.
#pragma once

#include <cstdint>
#include <utility>

#include "../../include/rarn.h"
#include "kv.cuh"

namespace rarn {
namespace check {

constexpr int64_t kMaxItems = int64_t(1) << 31;  // head rows of one call

inline bool type_ok(rarn_dtype d) { return d == RARN_F32 || d == RARN_F16 || d == RARN_BF16; }
inline int64_t size_of(rarn_dtype d) { return d == RARN_F32 ? 4 : 2; }
inline bool on(const void *p, unsigned a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// A byte range that repeats: `count` times every `stride` bytes, `extent`
// bytes each; the whole lies in [base, base + span).
struct Range {
    const char *base;
    int64_t span;
    int64_t stride, extent;  // stride 0: solid
};

inline Range solid(const void *p, int64_t bytes) {
    return Range{static_cast<const char *>(p), bytes, 0, 0};
}

// Whether two ranges can share a byte: their spans meet, and not as two
// repetitions of one stride that keep to their own parts of it (q, k and v
// inside one packed projection).
inline bool meet(const Range &a, const Range &b) {
    if (a.span <= 0 || b.span <= 0) return false;
    if (!(a.base < b.base + b.span && b.base < a.base + a.span)) return false;
    if (a.stride > 0 && a.stride == b.stride) {
        int64_t off = (b.base - a.base) % a.stride;
        if (off < 0) off += a.stride;
        if (off >= a.extent && off + b.extent <= a.stride) return false;
    }
    return true;
}

inline Range range_of(const rarn_heads &h, int64_t T, int64_t D) {
    const int64_t s = size_of(h.dtype), row = ((h.heads - 1) * h.head_stride + D) * s;
    Range r{static_cast<const char *>(h.data), (T - 1) * h.token_stride * s + row, 0, 0};
    if (T > 1 && h.token_stride * s >= row) {
        r.stride = h.token_stride * s;
        r.extent = row;
    }
    return r;
}

inline bool same(const rarn_heads &a, const rarn_heads &b) {
    return a.data == b.data && a.token_stride == b.token_stride && a.head_stride == b.head_stride;
}

// Whether `count` steps of `stride` stay within RARN_MAX_STRIDE, so that no
// offset below overflows (a single step is never taken).
inline bool reaches(int64_t stride, int64_t count) {
    return stride <= RARN_MAX_STRIDE && (count <= 1 || stride <= RARN_MAX_STRIDE / (count - 1));
}

// Sizes and strides of a [T, heads, D] matrix; an output's elements must not
// share memory among themselves.
inline rarn_status check_heads(const rarn_heads &h, int64_t T, int64_t D, bool output) {
    if (!type_ok(h.dtype) || h.heads < 1 || h.token_stride < 0 || h.head_stride < 0)
        return RARN_ERR_INVALID_ARG;
    if (h.heads > RARN_MAX_HEADS) return RARN_ERR_UNSUPPORTED;
    if (T == 0) return RARN_OK;
    if (!h.data) return RARN_ERR_INVALID_ARG;
    if (!reaches(h.token_stride, T) || h.head_stride > RARN_MAX_STRIDE)
        return RARN_ERR_UNSUPPORTED;
    if (!on(h.data, (unsigned)size_of(h.dtype))) return RARN_ERR_INVALID_ARG;
    if (output) {
        const bool by_token = (T == 1 || h.token_stride >= (h.heads - 1) * h.head_stride + D) &&
                              (h.heads == 1 || h.head_stride >= D);
        const bool by_head = (h.heads == 1 || h.head_stride >= (T - 1) * h.token_stride + D) &&
                             (T == 1 || h.token_stride >= D);
        if (!by_token && !by_head) return RARN_ERR_INVALID_ARG;
    }
    return RARN_OK;
}

// Whether every head of T tokens begins on an `a`-byte boundary.
inline bool packs_ok(const rarn_heads &h, int64_t T, int a = 16) {
    const int64_t s = size_of(h.dtype);
    return on(h.data, a) && (T == 1 || h.token_stride * s % a == 0) &&
           (h.heads == 1 || h.head_stride * s % a == 0);
}

// Whether the (stride, count) dimensions with `inner` units innermost address
// distinct units.
inline bool distinct(std::pair<int64_t, int64_t> (&d)[3], int64_t inner) {
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (d[j].first < d[i].first) std::swap(d[i], d[j]);
    int64_t reach = inner;
    for (auto &x : d) {
        if (x.second == 1) continue;
        if (x.first < reach) return false;
        reach = x.first * (x.second - 1) + reach;
    }
    return true;
}

struct CacheRanges {
    Range k, v, ks, vs;
};

inline rarn_status check_cache(const rarn_kv_cache *c, CacheRanges *out) {
    if (!c) return RARN_ERR_INVALID_ARG;
    if ((c->format != RARN_E4M3 && c->format != RARN_E5M2) ||
        (c->scale_mode != RARN_SCALE_TENSOR && c->scale_mode != RARN_SCALE_ROW))
        return RARN_ERR_INVALID_ARG;
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || c->num_pages < 1 || c->page_size < 1 ||
        c->heads < 1 || c->head_dim < 1)
        return RARN_ERR_INVALID_ARG;
    if (c->page_stride < 0 || c->head_stride < 0 || c->slot_stride < 0 ||
        c->scale_page_stride < 0 || c->scale_head_stride < 0 || c->scale_slot_stride < 0)
        return RARN_ERR_INVALID_ARG;
    if (c->head_dim % 16 || c->head_dim > 256 || c->heads > RARN_MAX_HEADS ||
        c->page_size > RARN_MAX_PAGE_SIZE || c->num_pages > (int64_t(1) << 31) - 1)
        return RARN_ERR_UNSUPPORTED;
    if (!reaches(c->page_stride, c->num_pages) || c->head_stride > RARN_MAX_STRIDE ||
        c->slot_stride > RARN_MAX_STRIDE || !reaches(c->scale_page_stride, c->num_pages) ||
        c->scale_head_stride > RARN_MAX_STRIDE || c->scale_slot_stride > RARN_MAX_STRIDE)
        return RARN_ERR_UNSUPPORTED;
    if (!on(c->k, 16) || !on(c->v, 16) || c->page_stride % 16 || c->head_stride % 16 ||
        c->slot_stride % 16)
        return RARN_ERR_UNSUPPORTED;
    if (!on(c->k_scale, 4) || !on(c->v_scale, 4)) return RARN_ERR_INVALID_ARG;
    std::pair<int64_t, int64_t> d[3] = {{c->page_stride, c->num_pages},
                                        {c->head_stride, c->heads},
                                        {c->slot_stride, c->page_size}};
    if (!distinct(d, c->head_dim)) return RARN_ERR_INVALID_ARG;
    const int64_t inside = (c->heads - 1) * c->head_stride +
                           (c->page_size - 1) * c->slot_stride + c->head_dim;
    const int64_t span = (c->num_pages - 1) * c->page_stride + inside;
    const bool by_page = c->num_pages > 1 && c->page_stride >= inside;
    out->k = Range{static_cast<const char *>(c->k), span, by_page ? c->page_stride : 0, inside};
    out->v = out->k;
    out->v.base = static_cast<const char *>(c->v);
    int64_t sspan = 4, sin = 0;
    bool s_by_page = false;
    if (c->scale_mode == RARN_SCALE_ROW) {
        std::pair<int64_t, int64_t> e[3] = {{c->scale_page_stride, c->num_pages},
                                            {c->scale_head_stride, c->heads},
                                            {c->scale_slot_stride, c->page_size}};
        if (!distinct(e, 1)) return RARN_ERR_INVALID_ARG;
        sin = ((c->heads - 1) * c->scale_head_stride + (c->page_size - 1) * c->scale_slot_stride +
               1) * 4;
        sspan = (c->num_pages - 1) * c->scale_page_stride * 4 + sin;
        s_by_page = c->num_pages > 1 && c->scale_page_stride * 4 >= sin;
    }
    out->ks = Range{reinterpret_cast<const char *>(c->k_scale), sspan,
                    s_by_page ? c->scale_page_stride * 4 : 0, sin};
    out->vs = out->ks;
    out->vs.base = reinterpret_cast<const char *>(c->v_scale);
    return RARN_OK;
}

inline kv::Cache view_of(const rarn_kv_cache &c) {
    kv::Cache v{};
    v.k = static_cast<uint8_t *>(c.k);
    v.v = static_cast<uint8_t *>(c.v);
    v.k_scale = c.k_scale;
    v.v_scale = c.v_scale;
    v.page_stride = c.page_stride;
    v.head_stride = c.head_stride;
    v.slot_stride = c.slot_stride;
    if (c.scale_mode == RARN_SCALE_ROW) {
        v.s_page = c.scale_page_stride;
        v.s_head = c.scale_head_stride;
        v.s_slot = c.scale_slot_stride;
    }
    v.pages = c.num_pages;
    v.page_size = c.page_size;
    v.heads = c.heads;
    v.fmt = c.format == RARN_E5M2 ? Q_E5M2 : Q_E4M3;
    v.mode = c.scale_mode == RARN_SCALE_ROW ? Q_ROW : Q_TENSOR;
    return v;
}

inline kv::Heads view_of(const rarn_heads &h) {
    return kv::Heads{h.data, h.token_stride, h.head_stride, h.heads};
}

// The page table of B sequences.
inline rarn_status check_table(const int32_t *table, int64_t stride, int64_t width, int64_t B) {
    if (B < 0 || width < 0 || stride < 0) return RARN_ERR_INVALID_ARG;
    if (B > RARN_MAX_SEQUENCES || width > (int64_t(1) << 31) - 1 || stride > RARN_MAX_STRIDE)
        return RARN_ERR_UNSUPPORTED;
    if (B > 0 && width > 0 && (!table || !on(table, 4))) return RARN_ERR_INVALID_ARG;
    return RARN_OK;
}

inline Range table_range(const int32_t *table, int64_t stride, int64_t width, int64_t B) {
    return solid(table, B > 0 && width > 0 ? ((B - 1) * stride + width) * 4 : 0);
}

}  // namespace check
}  // namespace rarn
