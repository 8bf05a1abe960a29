// pages_api.cu -- the C ABI of a step's pages and slots (rarn_kv_step, rarn_kv_trim)
// and of the cache's tidying behind an accepted path (rarn_kv_cache_compact).
// Argument checks come before anything is enqueued; no memory is allocated.
#include <algorithm>

#include "../../include/rarn.h"
#include "host.h"
#include "kv_check.h"
#include "pages.cuh"

using namespace rarn;
using namespace rarn::check;

namespace {

rarn_status check_pages(const rarn_kv_pages *g) {
    if (!g) return RARN_ERR_INVALID_ARG;
    if (g->sequences < 0 || g->table_width < 1 || g->table_stride < 0 || g->num_pages < 1 ||
        g->page_size < 1 || (g->sequences > 1 && g->table_stride < g->table_width))
        return RARN_ERR_INVALID_ARG;
    if (g->sequences > RARN_MAX_STEP_SEQUENCES || g->num_pages > (int64_t(1) << 31) - 1 ||
        g->page_size > RARN_MAX_PAGE_SIZE || !reaches(g->table_stride, g->sequences) ||
        g->table_width > ((int64_t(1) << 31) - 1) / g->page_size)
        return RARN_ERR_UNSUPPORTED;
    for (const void *p : {(const void *)g->free_pages, (const void *)g->free_count,
                          (const void *)g->ticket})
        if (!p || !on(p, 4)) return RARN_ERR_INVALID_ARG;
    // empty without sequences, and then often without an address
    for (const void *p : {(const void *)g->page_table, (const void *)g->held})
        if ((!p && g->sequences > 0) || !on(p, 4)) return RARN_ERR_INVALID_ARG;
    return RARN_OK;
}

// The ranges that a call on these pages writes.
struct PageRanges {
    Range r[5];
};

PageRanges ranges_of(const rarn_kv_pages &g) {
    const int64_t B = g.sequences;
    return PageRanges{{table_range(g.page_table, g.table_stride, g.table_width, B),
                       solid(g.held, B * 4), solid(g.free_pages, g.num_pages * 4),
                       solid(g.free_count, 4), solid(g.ticket, 4)}};
}

pages::Pool view_of(const rarn_kv_pages &g) {
    pages::Pool p{};
    p.table = g.page_table;
    p.table_stride = g.table_stride;
    p.held = g.held;
    p.free = g.free_pages;
    p.count = g.free_count;
    p.ticket = g.ticket;
    p.width = (int)g.table_width;
    p.num = (int)g.num_pages;
    p.page_size = g.page_size;
    p.B = (int)g.sequences;
    return p;
}

// No two of n ranges meet but inputs among themselves (the first `outs` are written).
bool apart(const Range *r, int outs, int n) {
    for (int i = 0; i < outs; ++i)
        for (int j = i + 1; j < n; ++j)
            if (meet(r[i], r[j])) return false;
    return true;
}

// The most dynamic shared memory of a call: k_step's two sums of every sequence.
constexpr int kMostSums = 2 * (RARN_MAX_STEP_SEQUENCES + 1) * 4;

template <typename P>
rarn_status launch(void (*kernel)(P), unsigned grid, size_t smem, const P &p, void *stream) {
    cudaError_t e = cudaSuccess;
    // The 48 KB that any kernel may have hold its static part too (some hundred bytes here).
    // The limit is always raised to the same value, so that no call lowers another's.
    if (smem > 47 * 1024)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSums);
    if (e == cudaSuccess)
        e = launch_kernel(kernel, dim3(grid), dim3(pages::kThreads), smem,
                          static_cast<cudaStream_t>(stream), host::pdl_enabled(), 1, p);
    return e == cudaSuccess ? RARN_OK : host::cuda_failed(e);
}

}  // namespace

extern "C" {

rarn_status rarn_kv_step(const rarn_kv_pages *pages, const int32_t *context_lens,
                         const int32_t *new_lens, int32_t *starts, int64_t *slots,
                         int64_t *positions, int32_t *served, int64_t tokens, void *stream) {
    rarn_status st = check_pages(pages);
    if (st != RARN_OK) return st;
    const int64_t B = pages->sequences;
    if (tokens < 0 || !starts || !on(starts, 4) || !served || !on(served, 4))
        return RARN_ERR_INVALID_ARG;
    if (tokens > (int64_t(1) << 31) - 1) return RARN_ERR_UNSUPPORTED;
    if (B > 0 && (!context_lens || !on(context_lens, 4) || !new_lens || !on(new_lens, 4)))
        return RARN_ERR_INVALID_ARG;
    if (tokens > 0 && (!slots || !on(slots, 8) || !positions || !on(positions, 8)))
        return RARN_ERR_INVALID_ARG;
    const PageRanges pr = ranges_of(*pages);
    Range r[11] = {pr.r[0], pr.r[1], pr.r[2], pr.r[3], pr.r[4], solid(starts, (B + 1) * 4),
                   solid(served, 4), solid(slots, tokens * 8), solid(positions, tokens * 8),
                   solid(context_lens, B * 4), solid(new_lens, B * 4)};
    if (!apart(r, 9, 11)) return RARN_ERR_ALIAS;
    host::Device dev;
    if ((st = host::current_device(&dev)) != RARN_OK) return st;
    pages::StepParams p{};
    p.pool = view_of(*pages);
    p.context = context_lens;
    p.fresh = new_lens;
    p.starts = starts;
    p.slots = slots;
    p.positions = positions;
    p.served = served;
    p.tokens = tokens;
    p.watchdog = dev.watchdog;
    const int64_t want = (tokens + pages::kThreads - 1) / pages::kThreads;
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(want, dev.num_sms * 4));
    return launch(pages::k_step, grid, (size_t)(2 * (B + 1) * 4), p, stream);
}

rarn_status rarn_kv_trim(const rarn_kv_pages *pages, const int32_t *lens, void *stream) {
    rarn_status st = check_pages(pages);
    if (st != RARN_OK) return st;
    const int64_t B = pages->sequences;
    if (B == 0) return RARN_OK;
    if (!lens || !on(lens, 4)) return RARN_ERR_INVALID_ARG;
    const PageRanges pr = ranges_of(*pages);
    Range r[6] = {pr.r[0], pr.r[1], pr.r[2], pr.r[3], pr.r[4], solid(lens, B * 4)};
    if (!apart(r, 5, 6)) return RARN_ERR_ALIAS;
    host::Device dev;
    if ((st = host::current_device(&dev)) != RARN_OK) return st;
    pages::TrimParams p{};
    p.pool = view_of(*pages);
    p.lens = lens;
    p.watchdog = dev.watchdog;
    const int64_t want = (pages->num_pages + 4 * pages::kThreads - 1) / (4 * pages::kThreads);
    return launch(pages::k_trim, (unsigned)std::min<int64_t>(want, 32), (size_t)((B + 1) * 4), p,
                  stream);
}

rarn_status rarn_kv_cache_compact(const rarn_kv_cache *cache, const int32_t *page_table,
                                  int64_t table_stride, int64_t table_width,
                                  const int32_t *context_lens, const int32_t *path,
                                  const int32_t *lengths, int64_t B, int64_t path_width,
                                  void *stream) {
    CacheRanges cr{};
    rarn_status st = check_cache(cache, &cr);
    if (st != RARN_OK) return st;
    if ((st = check_table(page_table, table_stride, table_width, B)) != RARN_OK) return st;
    if (path_width < 0) return RARN_ERR_INVALID_ARG;
    if (path_width > (1 << 24) || !reaches(table_stride, B)) return RARN_ERR_UNSUPPORTED;
    if (B == 0 || path_width <= 1) return RARN_OK;
    for (const void *p : {(const void *)context_lens, (const void *)path, (const void *)lengths})
        if (!p || !on(p, 4)) return RARN_ERR_INVALID_ARG;
    const bool rows = cache->scale_mode == RARN_SCALE_ROW;
    Range r[8] = {cr.k, cr.v, cr.ks, cr.vs, table_range(page_table, table_stride, table_width, B),
                  solid(context_lens, B * 4), solid(path, B * path_width * 4),
                  solid(lengths, B * 4)};
    if (!apart(r, rows ? 4 : 2, 8)) return RARN_ERR_ALIAS;
    const int64_t columns =
        2 * (int64_t)cache->heads * (cache->head_dim / 16) + (rows ? 2 * cache->heads : 0);
    const int64_t parts = (columns + pages::kMoveThreads - 1) / pages::kMoveThreads;
    if (B * parts > (int64_t(1) << 31) - 1) return RARN_ERR_UNSUPPORTED;
    host::Device dev;
    if ((st = host::current_device(&dev)) != RARN_OK) return st;
    pages::CompactParams p{};
    p.cache = check::view_of(*cache);
    p.table = page_table;
    p.table_stride = table_stride;
    p.width = (int)table_width;
    p.context = context_lens;
    p.path = path;
    p.lengths = lengths;
    p.W = (int)path_width;
    p.D = cache->head_dim;
    p.watchdog = dev.watchdog;
    const cudaError_t e = launch_kernel(pages::k_compact, dim3((unsigned)(B * parts)),
                                        dim3(pages::kMoveThreads), 0,
                                        static_cast<cudaStream_t>(stream), host::pdl_enabled(), 1,
                                        p, (int)parts);
    return e == cudaSuccess ? RARN_OK : host::cuda_failed(e);
}

}  // extern "C"
