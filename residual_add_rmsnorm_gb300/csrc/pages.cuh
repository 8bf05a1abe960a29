// pages.cuh -- a step's pages, slots and positions from the sequences' lengths, pages
// given back, and a tree's accepted tokens moved together in the cache.
//
// Integer work of a few kilobytes: what counts is one launch and few dependent
// loads.  Every CTA forms the prefix sums over all sequences by itself (in
// shared memory, 8 bytes a sequence), so that its rows need nothing from another
// CTA; what the sums were formed from (held, free_count) is written by the CTA
// that comes last, when no one reads it any more.
// Measured: a step and a trim of 8 sequences 5.7 us together, of 256 with 12 thousand
// new tokens 9.0; an accepted path's tokens moved in 256 sequences (8 heads of 128)
// 3.4 us, in one 3.0.
#pragma once

#include "kv.cuh"

namespace rarn {
namespace pages {

struct Pool {
    int32_t *table;       // [B, width]
    int64_t table_stride;
    int32_t *held;        // [B]: entries of each row that are pages
    int32_t *free;        // [num]: the first *count are free
    int32_t *count;
    unsigned int *ticket; // zero between calls
    int width, num, page_size, B;
};

struct StepParams {
    Pool pool;
    const int32_t *context, *fresh;  // [B]: cached and new tokens
    int32_t *starts;                 // [B + 1]
    int64_t *slots, *positions;      // [tokens]
    int32_t *served;
    int64_t tokens;
    unsigned int *watchdog;
};

struct TrimParams {
    Pool pool;
    const int32_t *lens;  // [B]
    unsigned int *watchdog;
};

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Exclusive sums over the CTA of two values a thread; the totals to every thread.
struct Sums {
    int64_t a, b;
};

__device__ __forceinline__ Sums warp_scan(Sums v) {  // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, v.a, m);
        const int64_t b = __shfl_up_sync(0xffffffffu, v.b, m);
        if (lane >= m) {
            v.a += a;
            v.b += b;
        }
    }
    return v;
}

__device__ __forceinline__ Sums block_scan(Sums v, Sums *red, Sums *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Sums in = warp_scan(v);
    if (lane == 31) red[warp] = in;
    __syncthreads();
    Sums before{0, 0}, all{0, 0};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) before = all;
        all.a += red[w].a;
        all.b += red[w].b;
    }
    *total = all;
    return Sums{before.a + in.a - v.a, before.b + in.b - v.b};
}

__device__ __forceinline__ int clamp31(int64_t v) {
    return v > INT32_MAX ? INT32_MAX : static_cast<int>(v);
}

// The last b with first[b] <= r, for first[0] <= r < first[n].
__device__ __forceinline__ int find(const int32_t *first, int n, int r) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= r) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Whether this CTA is the last to come here; then everything that the others read
// before has been read.  The ticket is back at zero.
__device__ __forceinline__ bool comes_last(unsigned int *ticket) {
    __shared__ bool last;
    __syncthreads();
    if (threadIdx.x == 0) {
        last = true;
        if (gridDim.x > 1) {
            __threadfence();
            last = atomicAdd(ticket, 1u) == gridDim.x - 1;
            if (last) *ticket = 0u;
            __threadfence();
        }
    }
    __syncthreads();
    return last;
}

// A sequence's new rows and the pages that they need beyond those held; rows < 0: its
// lengths or pages make no sense.
__device__ __forceinline__ Sums demand(const StepParams &p, int b) {
    const int64_t ctx = p.context[b], n = p.fresh[b], held = p.pool.held[b], ps = p.pool.page_size;
    if (n == 0) return Sums{0, 0};
    if (n < 0 || ctx < 0 || held < 0 || held > p.pool.width || held * ps < ctx ||
        ctx + n > p.pool.width * ps)
        return Sums{-1, 0};
    // below 2^31 + 2^20 by now
    const int need = (int)((uint32_t)(ctx + n + ps - 1) / (uint32_t)ps) - (int)held;
    return Sums{n, need > 0 ? need : 0};
}

// Sequences in order get rows and pages while both last: the first that would pass
// `tokens` rows or the free pages, and all behind it, get none.  The y-th new page
// of the call is free[count - 1 - y].
__global__ void __launch_bounds__(kThreads) k_step(const StepParams p) {
    extern __shared__ int32_t s_sums[];  // first[B + 1], pages[B + 1]
    __shared__ Sums red[kWarps];
    __shared__ int s_served;
    const int B = p.pool.B;
    int32_t *first = s_sums, *pre = s_sums + B + 1;
    grid_dependency_wait();
    grid_launch_dependents();
    if (threadIdx.x == 0) s_served = B;
    int count = *p.pool.count;
    const bool sound = count >= 0 && count <= p.pool.num;
    if (!sound) count = 0;
    // a thread's sequences are neighbours
    const int each = (B + kThreads - 1) / kThreads;
    const int b0 = min(B, (int)threadIdx.x * each), b1 = min(B, b0 + each);
    Sums mine{0, 0};
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        const Sums d = demand(p, b);
        bad |= d.a < 0;
        mine.a += d.a > 0 ? d.a : 0;
        mine.b += d.b;
    }
    Sums total;
    Sums at = block_scan(mine, red, &total);
    for (int b = b0; b < b1; ++b) {
        const Sums d = demand(p, b);
        first[b] = clamp31(at.a);
        pre[b] = clamp31(at.b);
        at.a += d.a > 0 ? d.a : 0;
        at.b += d.b;
        if (at.a > p.tokens || at.b > count) {
            atomicMin(&s_served, b);
            break;  // the sums do not fall
        }
    }
    if (threadIdx.x == 0) {
        first[B] = clamp31(total.a);
        pre[B] = clamp31(total.b);
    }
    __syncthreads();
    const int served = s_served, rows = first[served];
    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b <= B; b += kThreads)
            p.starts[b] = b <= served ? first[b] : rows;
        if (threadIdx.x == 0) *p.served = served;
        if (bad || !sound) atomicOr(p.watchdog, kv::kWatchIndex);
    }
    const int ps = p.pool.page_size;
    bool missing = false;
    for (int64_t r = (int64_t)blockIdx.x * kThreads + threadIdx.x; r < p.tokens;
         r += (int64_t)gridDim.x * kThreads) {
        int64_t slot = -1, pos = 0;
        if (r < rows) {
            const int b = find(first, served, (int)r);
            const int at = p.context[b] + ((int)r - first[b]);
            const int entry = at / ps, in = at - entry * ps, held = p.pool.held[b];
            int32_t *row = p.pool.table + b * p.pool.table_stride;
            int page;
            if (entry < held) {
                page = row[entry];
            } else {
                page = p.pool.free[count - 1 - (pre[b] + entry - held)];
                // a new page's first slot is a new token's: the held ones cover the context
                if (in == 0) row[entry] = page;
            }
            pos = at;
            if (page >= 0 && page < p.pool.num) slot = (int64_t)page * ps + in;
            else missing = true;
        }
        p.slots[r] = slot;
        p.positions[r] = pos;
    }
    if (missing) atomicOr(p.watchdog, kv::kWatchIndex);
    if (comes_last(p.pool.ticket)) {
        for (int b = threadIdx.x; b < served; b += kThreads) {
            const int need = pre[b + 1] - pre[b];
            if (need > 0) p.pool.held[b] += need;
        }
        if (threadIdx.x == 0 && sound) *p.pool.count = count - pre[served];
    }
}

// Every sequence keeps the pages of its first `lens` tokens; the x-th page given
// back, in order of sequences and their pages, becomes free[count' - 1 - x] with
// count' the new count: what k_step took for the same tokens, put back in its place.
__global__ void __launch_bounds__(kThreads) k_trim(const TrimParams p) {
    extern __shared__ int32_t s_sums[];  // pre[B + 1]
    __shared__ Sums red[kWarps];
    const int B = p.pool.B, ps = p.pool.page_size;
    int32_t *pre = s_sums;
    grid_dependency_wait();
    grid_launch_dependents();
    const int count = *p.pool.count;
    const int each = (B + kThreads - 1) / kThreads;
    const int b0 = min(B, (int)threadIdx.x * each), b1 = min(B, b0 + each);
    auto kept = [&](int b, int held) {
        const int n = p.lens[b];
        if (n < 0 || held < 0 || held > p.pool.width) return -1;
        return min(held, (int)(((uint32_t)n + (uint32_t)ps - 1) / (uint32_t)ps));
    };
    Sums mine{0, 0}, total;
    for (int b = b0; b < b1; ++b) {
        const int held = p.pool.held[b], keep = kept(b, held);
        if (keep < 0) mine.b = 1;
        else mine.a += held - keep;
    }
    Sums at = block_scan(mine, red, &total);
    const bool sound = count >= 0 && count <= p.pool.num && total.a <= p.pool.num - count;
    if ((total.b > 0 || !sound) && blockIdx.x == 0 && threadIdx.x == 0)
        atomicOr(p.watchdog, kv::kWatchIndex);
    if (!sound) {  // every CTA alike: more pages than there are, nothing is moved
        comes_last(p.pool.ticket);
        return;
    }
    for (int b = b0; b < b1; ++b) {
        const int held = p.pool.held[b], keep = kept(b, held);
        pre[b] = (int)at.a;
        if (keep >= 0) at.a += held - keep;
    }
    if (threadIdx.x == 0) pre[B] = (int)total.a;
    __syncthreads();
    const int gone = (int)total.a;
    bool missing = false;
    for (int64_t x = (int64_t)blockIdx.x * kThreads + threadIdx.x; x < gone;
         x += (int64_t)gridDim.x * kThreads) {
        const int b = find(pre, B, (int)x);
        const int entry = kept(b, p.pool.held[b]) + ((int)x - pre[b]);
        int32_t *e = p.pool.table + b * p.pool.table_stride + entry;
        const int page = *e;
        missing |= page < 0 || page >= p.pool.num;
        p.pool.free[count + gone - 1 - x] = page;
        *e = -1;
    }
    if (missing) atomicOr(p.watchdog, kv::kWatchIndex);
    if (comes_last(p.pool.ticket)) {
        for (int b = threadIdx.x; b < B; b += kThreads) {
            const int n = pre[b + 1] - pre[b];
            if (n > 0) p.pool.held[b] -= n;
        }
        if (threadIdx.x == 0) *p.pool.count = count + gone;
    }
}

struct CompactParams {
    kv::Cache cache;
    const int32_t *table;   // [B, width]
    int64_t table_stride;
    int width;
    const int32_t *context; // [B]
    const int32_t *path;    // [B, W]
    const int32_t *lengths; // [B]
    int W, D;
    unsigned int *watchdog;
};

constexpr int kMoveThreads = 128;
constexpr int kMoveRows = 32;

// Token context + path[j] goes to context + j, j = 1 .. length - 1.  A path rises, so
// that no row goes where a later one comes from: a thread takes one 16-byte
// piece (or one scale) of all rows in order, a few rows loaded ahead of their
// stores, and needs no other thread.
__global__ void __launch_bounds__(kMoveThreads) k_compact(const CompactParams p, int parts) {
    __shared__ int64_t s_from[kMoveRows], s_to[kMoveRows];    // code offsets; from < 0: stays
    __shared__ int64_t s_sfrom[kMoveRows], s_sto[kMoveRows];  // scale offsets
    __shared__ int s_stop;
    grid_dependency_wait();
    grid_launch_dependents();
    const int b = blockIdx.x / parts, part = blockIdx.x - b * parts;
    int n = p.lengths[b];
    const int64_t ctx = p.context[b];
    const bool reporter = part == 0;
    if (n > p.W || ctx < 0) {
        if (reporter && threadIdx.x == 0) atomicOr(p.watchdog, kv::kWatchIndex);
        if (ctx < 0) return;
        n = p.W;
    }
    const int pieces = p.D / 16, codes = 2 * p.cache.heads * pieces;
    const int columns = codes + (p.cache.mode == Q_ROW ? 2 * p.cache.heads : 0);
    const int c = part * kMoveThreads + threadIdx.x;
    const bool is_code = c < codes, is_scale = !is_code && c < columns;
    const int hp = is_code ? c / pieces : c - codes;
    const bool val = hp >= p.cache.heads;
    const int head = val ? hp - p.cache.heads : hp;
    uint8_t *code = (val ? p.cache.v : p.cache.k) + head * p.cache.head_stride +
                    (is_code ? c - hp * pieces : 0) * 16;
    float *scale = (val ? p.cache.v_scale : p.cache.k_scale) + head * p.cache.s_head;
    const int32_t *path = p.path + (int64_t)b * p.W;
    const int32_t *table = p.table + b * p.table_stride;

    for (int j0 = 1; j0 < n; j0 += kMoveRows) {
        if (threadIdx.x < 32) {
            const int j = j0 + threadIdx.x;
            int64_t from = -1, to = 0, sfrom = 0, sto = 0;
            bool rises = true, lost = false;
            if (j < n) {
                const int at = path[j], before = path[j - 1];
                rises = before >= j - 1 && at > before;
                if (rises && at > j) {
                    auto place = [&](int64_t t, int64_t *code_at, int64_t *scale_at) {
                        const uint32_t entry = (uint32_t)t / (uint32_t)p.cache.page_size;
                        if (entry >= (uint32_t)p.width) return false;
                        const int page = table[entry];
                        if (page < 0 || page >= p.cache.pages) return false;
                        const int64_t in = (uint32_t)t - entry * (uint32_t)p.cache.page_size;
                        *code_at = page * p.cache.page_stride + in * p.cache.slot_stride;
                        *scale_at = page * p.cache.s_page + in * p.cache.s_slot;
                        return true;
                    };
                    lost = !place(ctx + at, &from, &sfrom) || !place(ctx + j, &to, &sto);
                    if (lost) from = -1;
                }
            }
            const unsigned fell = __ballot_sync(0xffffffffu, !rises);
            const int stop = fell ? __ffs(fell) - 1 : 32;  // nothing moves from there on
            if ((int)threadIdx.x >= stop) from = -1;
            if (reporter && (lost || (!rises && (int)threadIdx.x == stop)))
                atomicOr(p.watchdog, kv::kWatchIndex);
            s_from[threadIdx.x] = from;
            s_to[threadIdx.x] = to;
            s_sfrom[threadIdx.x] = sfrom;
            s_sto[threadIdx.x] = sto;
            if (threadIdx.x == 0) s_stop = fell != 0;
        }
        __syncthreads();
        const int rows = min(kMoveRows, n - j0);
        constexpr int U = 4;
        for (int i0 = 0; i0 < rows; i0 += U) {
            uint4 w[U];
            float s[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u;
                if (i >= rows || s_from[i] < 0) continue;
                if (is_code) w[u] = ld_stream(code + s_from[i]);
                else if (is_scale) s[u] = scale[s_sfrom[i]];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u;
                if (i >= rows || s_from[i] < 0) continue;
                if (is_code) st_global(code + s_to[i], w[u]);
                else if (is_scale) scale[s_sto[i]] = s[u];
            }
        }
        const bool stop = s_stop;
        __syncthreads();
        if (stop) return;
    }
}

}  // namespace pages
}  // namespace rarn
