// kv_api.cu -- the C ABI's attention side: per-head norm and rotation, the
// 8-bit key / value cache, attention of drafted tokens over it.  Argument
// checks come before anything is enqueued; no memory is allocated.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <utility>

#include "../../include/rarn.h"
#include "host.h"
#include "kv_rows.cuh"
#include "tree_attn.cuh"
#include "tree_plan.h"

namespace rarn {
namespace kv {
// instantiated in kv_rows_{bf16,f16,f32}.cu
extern template cudaError_t launch_head_rows<__nv_bfloat16>(const RowParams &, bool, int, bool,
                                                            cudaStream_t);
extern template cudaError_t launch_head_rows<__half>(const RowParams &, bool, int, bool,
                                                     cudaStream_t);
extern template cudaError_t launch_head_rows<float>(const RowParams &, bool, int, bool,
                                                    cudaStream_t);
extern template cudaError_t launch_cache_read<__nv_bfloat16>(const ReadParams &, int, int, bool,
                                                             cudaStream_t);
extern template cudaError_t launch_cache_read<__half>(const ReadParams &, int, int, bool,
                                                      cudaStream_t);
extern template cudaError_t launch_cache_read<float>(const ReadParams &, int, int, bool,
                                                     cudaStream_t);
}  // namespace kv
namespace tree {
// instantiated in tree_attn_{e4m3,e5m2}.cu
template <bool kE5M2>
cudaError_t launch_tree(const Params &, const Plan &, int, bool, cudaStream_t);
extern template cudaError_t launch_tree<false>(const Params &, const Plan &, int, bool,
                                               cudaStream_t);
extern template cudaError_t launch_tree<true>(const Params &, const Plan &, int, bool,
                                              cudaStream_t);
}  // namespace tree
}  // namespace rarn

using namespace rarn;

namespace {

constexpr int64_t kMaxItems = int64_t(1) << 31;  // head rows of one call

bool type_ok(rarn_dtype d) { return d == RARN_F32 || d == RARN_F16 || d == RARN_BF16; }
int64_t size_of(rarn_dtype d) { return d == RARN_F32 ? 4 : 2; }
bool on(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A byte range that repeats: `count` times every `stride` bytes, `extent`
// bytes each; the whole lies in [base, base + span).
struct Range {
    const char *base;
    int64_t span;
    int64_t stride, extent;  // stride 0: solid
};

Range solid(const void *p, int64_t bytes) {
    return Range{static_cast<const char *>(p), bytes, 0, 0};
}

// Whether two ranges can share a byte: their spans meet, and not as two
// repetitions of one stride that keep to their own parts of it (q, k and v
// inside one packed projection).
bool meet(const Range &a, const Range &b) {
    if (a.span <= 0 || b.span <= 0) return false;
    if (!(a.base < b.base + b.span && b.base < a.base + a.span)) return false;
    if (a.stride > 0 && a.stride == b.stride) {
        int64_t off = (b.base - a.base) % a.stride;
        if (off < 0) off += a.stride;
        if (off >= a.extent && off + b.extent <= a.stride) return false;
    }
    return true;
}

Range range_of(const rarn_heads &h, int64_t T, int64_t D) {
    const int64_t s = size_of(h.dtype), row = ((h.heads - 1) * h.head_stride + D) * s;
    Range r{static_cast<const char *>(h.data), (T - 1) * h.token_stride * s + row, 0, 0};
    if (T > 1 && h.token_stride * s >= row) {
        r.stride = h.token_stride * s;
        r.extent = row;
    }
    return r;
}

bool same(const rarn_heads &a, const rarn_heads &b) {
    return a.data == b.data && a.token_stride == b.token_stride && a.head_stride == b.head_stride;
}

// Whether `count` steps of `stride` stay within RARN_MAX_STRIDE, so that no
// offset below overflows (a single step is never taken).
bool reaches(int64_t stride, int64_t count) {
    return stride <= RARN_MAX_STRIDE && (count <= 1 || stride <= RARN_MAX_STRIDE / (count - 1));
}

// Sizes and strides of a [T, heads, D] matrix; an output's elements must not
// share memory among themselves.
rarn_status check_heads(const rarn_heads &h, int64_t T, int64_t D, bool output) {
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
bool packs_ok(const rarn_heads &h, int64_t T, int a = 16) {
    const int64_t s = size_of(h.dtype);
    return on(h.data, a) && (T == 1 || h.token_stride * s % a == 0) &&
           (h.heads == 1 || h.head_stride * s % a == 0);
}

// Whether the (stride, count) dimensions with `inner` units innermost address
// distinct units.
bool distinct(std::pair<int64_t, int64_t> (&d)[3], int64_t inner) {
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

rarn_status check_cache(const rarn_kv_cache *c, CacheRanges *out) {
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

kv::Cache view_of(const rarn_kv_cache &c) {
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

kv::Heads view_of(const rarn_heads &h) {
    return kv::Heads{h.data, h.token_stride, h.head_stride, h.heads};
}

rarn_status check_rotation(const rarn_rotation *r, int64_t T, int64_t D) {
    if (!r) return RARN_OK;
    if (r->style != RARN_ROTATE_HALF && r->style != RARN_ROTATE_INTERLEAVED)
        return RARN_ERR_INVALID_ARG;
    if (r->rot_dim < 2 || r->rot_dim % 2 || r->rot_dim > D || r->table_rows < 1)
        return RARN_ERR_INVALID_ARG;
    if (r->table_rows > RARN_MAX_STRIDE) return RARN_ERR_UNSUPPORTED;
    if (T > 0 && (!r->cos_sin || !r->positions)) return RARN_ERR_INVALID_ARG;
    if (!on(r->cos_sin, 4) || !on(r->positions, 8)) return RARN_ERR_INVALID_ARG;
    return RARN_OK;
}

// Checks, then launches, the rows of a call: q and k normalised and rotated,
// k and v into the cache.  Absent parts have heads == 0 / null pointers.
struct RowCall {
    rarn_heads q_out{}, k_out{}, q{}, k{}, v{};
    const void *q_gamma = nullptr, *k_gamma = nullptr;
    const rarn_rotation *rot = nullptr;
    const rarn_kv_cache *cache = nullptr;
    const int64_t *slots = nullptr;
    bool has_q = false, has_k_out = false, has_v = false;
    int64_t T = 0, D = 0;
    float eps = 0.f;
};

rarn_status run_rows(const RowCall &c, void *stream) {
    if (c.T < 0 || c.D < 1 || !(c.eps >= 0.f) || std::isinf(c.eps)) return RARN_ERR_INVALID_ARG;
    rarn_status st;
    CacheRanges cr{};
    if (c.cache && (st = check_cache(c.cache, &cr)) != RARN_OK) return st;
    const rarn_dtype dt = c.k.dtype;
    if ((st = check_heads(c.k, c.T, c.D, false)) != RARN_OK) return st;
    if (c.has_q) {
        if ((st = check_heads(c.q, c.T, c.D, false)) != RARN_OK) return st;
        if ((st = check_heads(c.q_out, c.T, c.D, true)) != RARN_OK) return st;
        if (c.q_out.heads != c.q.heads) return RARN_ERR_INVALID_ARG;
        if (c.q.dtype != dt || c.q_out.dtype != dt) return RARN_ERR_UNSUPPORTED;
    }
    if (c.has_k_out) {
        if ((st = check_heads(c.k_out, c.T, c.D, true)) != RARN_OK) return st;
        if (c.k_out.heads != c.k.heads) return RARN_ERR_INVALID_ARG;
        if (c.k_out.dtype != dt) return RARN_ERR_UNSUPPORTED;
    }
    if (c.has_v) {
        if ((st = check_heads(c.v, c.T, c.D, false)) != RARN_OK) return st;
        if (c.v.heads != c.k.heads) return RARN_ERR_INVALID_ARG;
        if (c.v.dtype != dt) return RARN_ERR_UNSUPPORTED;
    }
    if (c.cache && (c.cache->heads != c.k.heads || c.cache->head_dim != c.D))
        return RARN_ERR_INVALID_ARG;
    if ((st = check_rotation(c.rot, c.T, c.D)) != RARN_OK) return st;
    if (c.T == 0) return RARN_OK;
    if (c.cache && (!c.slots || !on(c.slots, 8))) return RARN_ERR_INVALID_ARG;
    const int64_t heads = (c.has_q ? c.q.heads : 0) + c.k.heads + (c.has_v ? c.v.heads : 0);
    if (c.D > RARN_MAX_HEAD_DIM || c.T >= kMaxItems / heads) return RARN_ERR_UNSUPPORTED;
    const int64_t s = size_of(dt);
    if (!on(c.q_gamma, (unsigned)s) || !on(c.k_gamma, (unsigned)s)) return RARN_ERR_INVALID_ARG;

    // outputs against everything, an in-place q or k apart
    Range outs[6], ins[9];
    int no = 0, ni = 0;
    if (c.has_q) outs[no++] = range_of(c.q_out, c.T, c.D);
    if (c.has_k_out) outs[no++] = range_of(c.k_out, c.T, c.D);
    const int row_outs = no;
    if (c.cache) {
        outs[no++] = cr.k;
        outs[no++] = cr.v;
        if (c.cache->scale_mode == RARN_SCALE_ROW) {
            outs[no++] = cr.ks;
            outs[no++] = cr.vs;
        } else {
            ins[ni++] = cr.ks;
            ins[ni++] = cr.vs;
        }
        ins[ni++] = solid(c.slots, c.T * 8);
    }
    if (c.q_gamma) ins[ni++] = solid(c.q_gamma, c.D * s);
    if (c.k_gamma) ins[ni++] = solid(c.k_gamma, c.D * s);
    if (c.rot) {
        ins[ni++] = solid(c.rot->cos_sin, c.rot->table_rows * c.rot->rot_dim * 4);
        ins[ni++] = solid(c.rot->positions, c.T * 8);
    }
    for (int i = 0; i < no; ++i) {
        for (int j = i + 1; j < no; ++j)
            if (meet(outs[i], outs[j])) return RARN_ERR_ALIAS;
        for (int j = 0; j < ni; ++j)
            if (meet(outs[i], ins[j])) return RARN_ERR_ALIAS;
        const bool is_q = c.has_q && i == 0, is_k = c.has_k_out && i == row_outs - 1 && i < row_outs;
        if (c.has_q && !(is_q && same(c.q, c.q_out)) && meet(outs[i], range_of(c.q, c.T, c.D)))
            return RARN_ERR_ALIAS;
        if (!(is_k && same(c.k, c.k_out)) && meet(outs[i], range_of(c.k, c.T, c.D)))
            return RARN_ERR_ALIAS;
        if (c.has_v && meet(outs[i], range_of(c.v, c.T, c.D))) return RARN_ERR_ALIAS;
    }

    host::Device dev;
    if ((st = host::current_device(&dev)) != RARN_OK) return st;
    kv::RowParams p{};
    if (c.has_q) {
        p.q = view_of(c.q);
        p.q_out = view_of(c.q_out);
    }
    p.k = view_of(c.k);
    if (c.has_k_out) p.k_out = view_of(c.k_out);
    if (c.has_v) p.v = view_of(c.v);
    p.q_gamma = c.q_gamma;
    p.k_gamma = c.k_gamma;
    if (c.rot) {
        p.table = c.rot->cos_sin;
        p.positions = c.rot->positions;
        p.table_rows = c.rot->table_rows;
        p.rot = c.rot->rot_dim;
        p.interleaved = c.rot->style == RARN_ROTATE_INTERLEAVED;
    }
    if (c.cache) {
        p.cache = view_of(*c.cache);
        p.slots = c.slots;
    }
    p.T = c.T;
    p.D = (int)c.D;
    p.eps = c.eps;
    p.watchdog = dev.watchdog;
    // the vector kernel: 16-byte packs throughout, both packs of a lane on one
    // side of the rotation's end
    const int64_t e = 16 / s;
    bool vec = c.D % (2 * e) == 0 && c.D / (2 * e) <= 32 && packs_ok(c.k, c.T) &&
               (!c.q_gamma || on(c.q_gamma, 16)) && (!c.k_gamma || on(c.k_gamma, 16));
    if (c.has_q) vec = vec && packs_ok(c.q, c.T) && packs_ok(c.q_out, c.T);
    if (c.has_k_out) vec = vec && packs_ok(c.k_out, c.T);
    if (c.has_v) vec = vec && packs_ok(c.v, c.T);
    if (c.rot) vec = vec && c.rot->rot_dim % (2 * e) == 0 && on(c.rot->cos_sin, 16);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool pdl = host::pdl_enabled();
    cudaError_t err;
    switch (dt) {
    case RARN_BF16: err = kv::launch_head_rows<__nv_bfloat16>(p, vec, dev.num_sms, pdl, cs); break;
    case RARN_F16: err = kv::launch_head_rows<__half>(p, vec, dev.num_sms, pdl, cs); break;
    default: err = kv::launch_head_rows<float>(p, vec, dev.num_sms, pdl, cs); break;
    }
    return err == cudaSuccess ? RARN_OK : host::cuda_failed(err);
}

// The page table of B sequences.
rarn_status check_table(const int32_t *table, int64_t stride, int64_t width, int64_t B) {
    if (B < 0 || width < 0 || stride < 0) return RARN_ERR_INVALID_ARG;
    if (B > RARN_MAX_SEQUENCES || width > (int64_t(1) << 31) - 1 || stride > RARN_MAX_STRIDE)
        return RARN_ERR_UNSUPPORTED;
    if (B > 0 && width > 0 && (!table || !on(table, 4))) return RARN_ERR_INVALID_ARG;
    return RARN_OK;
}

Range table_range(const int32_t *table, int64_t stride, int64_t width, int64_t B) {
    return solid(table, B > 0 && width > 0 ? ((B - 1) * stride + width) * 4 : 0);
}

}  // namespace

extern "C" {

rarn_status rarn_qk_norm_rope(rarn_heads q_out, rarn_heads k_out, rarn_heads q, rarn_heads k,
                              const void *q_gamma, const void *k_gamma,
                              const rarn_rotation *rotation, int64_t T, int64_t D, float eps,
                              void *stream) {
    RowCall c;
    c.q_out = q_out;
    c.k_out = k_out;
    c.q = q;
    c.k = k;
    c.q_gamma = q_gamma;
    c.k_gamma = k_gamma;
    c.rot = rotation;
    c.has_q = c.has_k_out = true;
    c.T = T;
    c.D = D;
    c.eps = eps;
    return run_rows(c, stream);
}

rarn_status rarn_kv_cache_write(const rarn_kv_cache *cache, rarn_heads k, rarn_heads v,
                                const int64_t *slots, int64_t T, void *stream) {
    if (!cache) return RARN_ERR_INVALID_ARG;
    RowCall c;
    c.k = k;
    c.v = v;
    c.cache = cache;
    c.slots = slots;
    c.has_v = true;
    c.T = T;
    c.D = cache->head_dim;
    return run_rows(c, stream);
}

rarn_status rarn_qk_norm_rope_kv_write(rarn_heads q_out, const rarn_kv_cache *cache, rarn_heads q,
                                       rarn_heads k, rarn_heads v, const void *q_gamma,
                                       const void *k_gamma, const rarn_rotation *rotation,
                                       const int64_t *slots, int64_t T, float eps, void *stream) {
    if (!cache) return RARN_ERR_INVALID_ARG;
    RowCall c;
    c.q_out = q_out;
    c.q = q;
    c.k = k;
    c.v = v;
    c.q_gamma = q_gamma;
    c.k_gamma = k_gamma;
    c.rot = rotation;
    c.cache = cache;
    c.slots = slots;
    c.has_q = c.has_v = true;
    c.T = T;
    c.D = cache->head_dim;
    c.eps = eps;
    return run_rows(c, stream);
}

rarn_status rarn_kv_cache_read(rarn_heads k_out, rarn_heads v_out, const rarn_kv_cache *cache,
                               const int32_t *page_table, int64_t table_stride,
                               int64_t table_width, const int32_t *starts, int64_t B,
                               int64_t rows, void *stream) {
    CacheRanges cr{};
    rarn_status st = check_cache(cache, &cr);
    if (st != RARN_OK) return st;
    if (rows < 0) return RARN_ERR_INVALID_ARG;
    if ((st = check_table(page_table, table_stride, table_width, B)) != RARN_OK) return st;
    const int64_t D = cache->head_dim;
    if ((st = check_heads(k_out, rows, D, true)) != RARN_OK) return st;
    if ((st = check_heads(v_out, rows, D, true)) != RARN_OK) return st;
    if (k_out.heads != cache->heads || v_out.heads != cache->heads) return RARN_ERR_INVALID_ARG;
    if (k_out.dtype != v_out.dtype) return RARN_ERR_UNSUPPORTED;
    if (rows == 0 || B == 0) return RARN_OK;
    if (!starts || !on(starts, 4)) return RARN_ERR_INVALID_ARG;
    if (rows >= kMaxItems) return RARN_ERR_UNSUPPORTED;
    const Range outs[2] = {range_of(k_out, rows, D), range_of(v_out, rows, D)};
    const Range ins[6] = {cr.k, cr.v, cr.ks, cr.vs,
                          table_range(page_table, table_stride, table_width, B),
                          solid(starts, (B + 1) * 4)};
    if (meet(outs[0], outs[1])) return RARN_ERR_ALIAS;
    for (const Range &o : outs)
        for (const Range &i : ins)
            if (meet(o, i)) return RARN_ERR_ALIAS;
    host::Device dev;
    if ((st = host::current_device(&dev)) != RARN_OK) return st;
    kv::ReadParams p{};
    p.k_out = view_of(k_out);
    p.v_out = view_of(v_out);
    p.cache = view_of(*cache);
    p.table = page_table;
    p.table_stride = table_stride;
    p.table_width = (int)table_width;
    p.starts = starts;
    p.B = (int)B;
    p.rows = rows;
    p.D = (int)D;
    p.watchdog = dev.watchdog;
    const bool vec = packs_ok(k_out, rows) && packs_ok(v_out, rows);
    const int store = !vec ? 0 : packs_ok(k_out, rows, 32) && packs_ok(v_out, rows, 32) ? 32 : 16;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool pdl = host::pdl_enabled();
    cudaError_t e;
    switch (k_out.dtype) {
    case RARN_BF16: e = kv::launch_cache_read<__nv_bfloat16>(p, store, dev.num_sms, pdl, cs); break;
    case RARN_F16: e = kv::launch_cache_read<__half>(p, store, dev.num_sms, pdl, cs); break;
    default: e = kv::launch_cache_read<float>(p, store, dev.num_sms, pdl, cs); break;
    }
    return e == cudaSuccess ? RARN_OK : host::cuda_failed(e);
}

int64_t rarn_tree_attention_workspace_bytes(int64_t tokens, int64_t B, int64_t q_heads,
                                            int64_t kv_heads, int64_t D) {
    if (tokens < 0 || B < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads ||
        q_heads > RARN_MAX_HEADS || B > RARN_MAX_SEQUENCES || !tree::dim_ok(D) ||
        tokens >= kMaxItems / q_heads)
        return -1;
    if (tokens == 0 || B == 0) return 0;
    const tree::Plan a = tree::plan(tokens, B, q_heads, kv_heads, D, false),
                     b = tree::plan(tokens, B, q_heads, kv_heads, D, true);
    return a.segments < kMaxItems ? std::max(a.bytes, b.bytes) : -1;
}

rarn_status rarn_plan_tree_attention(int64_t tokens, int64_t B, int64_t q_heads, int64_t kv_heads,
                                     int64_t D, int64_t page_size, char *out, size_t cap) {
    if (!out || cap == 0 || tokens < 0 || B < 0 || q_heads < 1 || kv_heads < 1 || page_size < 1)
        return RARN_ERR_INVALID_ARG;
    if (page_size > RARN_MAX_PAGE_SIZE ||
        rarn_tree_attention_workspace_bytes(tokens, B, q_heads, kv_heads, D) < 0) {
        snprintf(out, cap, "none: unsupported sizes");
        return RARN_ERR_UNSUPPORTED;
    }
    if (tokens == 0 || B == 0) {
        snprintf(out, cap, "none: no rows");
        return RARN_OK;
    }
    const tree::Plan pl = tree::plan(tokens, B, q_heads, kv_heads, D,
                                     page_size % tree::kBoxSlots == 0);
    snprintf(out, cap, "tree.%s rows=%d", pl.tiles ? "tiles" : "rows", pl.rows);
    return RARN_OK;
}

rarn_status rarn_tree_attention(rarn_heads out, rarn_heads q, const rarn_kv_cache *cache,
                                const int32_t *page_table, int64_t table_stride,
                                int64_t table_width, const int32_t *context_lens,
                                const int32_t *starts, const int32_t *mask, int64_t mask_words,
                                int64_t B, int64_t tokens, float scale, void *workspace,
                                size_t workspace_bytes, void *stream) {
    CacheRanges cr{};
    rarn_status st = check_cache(cache, &cr);
    if (st != RARN_OK) return st;
    if (tokens < 0 || !(scale > 0.f) || std::isinf(scale) || mask_words < 0)
        return RARN_ERR_INVALID_ARG;
    if ((st = check_table(page_table, table_stride, table_width, B)) != RARN_OK) return st;
    const int64_t D = cache->head_dim;
    if ((st = check_heads(q, tokens, D, false)) != RARN_OK) return st;
    if ((st = check_heads(out, tokens, D, true)) != RARN_OK) return st;
    if (q.heads != out.heads || q.heads % cache->heads) return RARN_ERR_INVALID_ARG;
    if (q.dtype != out.dtype || q.dtype == RARN_F32 || !tree::dim_ok(D))
        return RARN_ERR_UNSUPPORTED;
    if (mask && (mask_words < 1 || !on(mask, 4))) return RARN_ERR_INVALID_ARG;
    if (mask_words > RARN_MAX_MASK_WORDS) return RARN_ERR_UNSUPPORTED;
    if (tokens == 0 || B == 0) return RARN_OK;
    if (!context_lens || !starts || !on(context_lens, 4) || !on(starts, 4))
        return RARN_ERR_INVALID_ARG;
    if (tokens >= kMaxItems / q.heads || !packs_ok(q, tokens)) return RARN_ERR_UNSUPPORTED;
    // keys are counted in 32 bits, with room for a tile behind the last
    if (table_width > ((int64_t(1) << 31) - 4096) / cache->page_size) return RARN_ERR_UNSUPPORTED;
    const tree::Plan pl =
        tree::plan(tokens, B, q.heads, cache->heads, D, cache->page_size % tree::kBoxSlots == 0);
    if (pl.segments >= kMaxItems) return RARN_ERR_UNSUPPORTED;
    if (!workspace || !on(workspace, 32) ||
        (int64_t)workspace_bytes <
            rarn_tree_attention_workspace_bytes(tokens, B, q.heads, cache->heads, D))
        return RARN_ERR_INVALID_ARG;
    const Range outs[2] = {range_of(out, tokens, D), solid(workspace, pl.bytes)};
    const Range ins[8] = {range_of(q, tokens, D), cr.k, cr.v, cr.ks, cr.vs,
                          table_range(page_table, table_stride, table_width, B),
                          solid(context_lens, B * 4), solid(starts, (B + 1) * 4)};
    if (meet(outs[0], outs[1])) return RARN_ERR_ALIAS;
    for (const Range &o : outs) {
        for (const Range &i : ins)
            if (meet(o, i)) return RARN_ERR_ALIAS;
        if (mask && meet(o, solid(mask, tokens * mask_words * 4))) return RARN_ERR_ALIAS;
    }
    host::Device dev;
    if ((st = host::current_device(&dev)) != RARN_OK) return st;
    tree::Params p{};
    p.q = view_of(q);
    p.out = view_of(out);
    p.cache = view_of(*cache);
    p.table = page_table;
    p.table_stride = table_stride;
    p.table_width = (int)table_width;
    p.context = context_lens;
    p.starts = starts;
    p.mask = reinterpret_cast<const uint32_t *>(mask);
    p.words = (int)mask_words;
    p.B = (int)B;
    p.tokens = tokens;
    p.D = (int)D;
    p.G = q.heads / cache->heads;
    p.bf16 = q.dtype == RARN_BF16;
    p.out_aligned = on(out.data, 8) && out.token_stride % 4 == 0 && out.head_stride % 4 == 0;
    p.scale_log2 = scale * 1.44269504088896340736f;
    const int ps = cache->page_size;
    p.whole_steps =
        ps % tree::kStep == 0 &&
        (cache->scale_mode == RARN_SCALE_TENSOR ||
         (on(cache->k_scale, 16) && on(cache->v_scale, 16) && cache->scale_slot_stride == 1 &&
          (cache->heads == 1 || cache->scale_head_stride % 4 == 0) &&
          (cache->num_pages == 1 || cache->scale_page_stride % 4 == 0)));
    p.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (ps == 1 << i) p.page_shift = i;
    char *ws = static_cast<char *>(workspace);
    p.count = reinterpret_cast<int *>(ws);
    p.joins = reinterpret_cast<tree::Join *>(ws + pl.joins_off);
    p.ml = reinterpret_cast<float2 *>(ws + pl.ml_off);
    p.part = reinterpret_cast<float *>(ws + pl.part_off);
    p.max_segs = (int)pl.segments;
    p.watchdog = dev.watchdog;
    p.wait_limit_ns = tree::kWaitLimitNs;
    p.stall_fill = -1;
    long long fill;
    if ((pl.tiles || (p.whole_steps && tree::rows_by_tma(D))) &&
        host::take_stall(&fill, &p.wait_limit_ns))
        p.stall_fill = (int)std::min<long long>(fill, INT32_MAX);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool pdl = host::pdl_enabled();
    const cudaError_t e = cache->format == RARN_E5M2
                              ? tree::launch_tree<true>(p, pl, dev.num_sms, pdl, cs)
                              : tree::launch_tree<false>(p, pl, dev.num_sms, pdl, cs);
    return e == cudaSuccess ? RARN_OK : host::cuda_failed(e);
}

}  // extern "C"
