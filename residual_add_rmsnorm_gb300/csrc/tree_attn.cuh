// tree_attn.cuh -- attention of drafted tokens over the paged 8-bit cache.
//
//   s_ij = scale * (q_i . K_j) * ks_j          over the visible j
//   o_i  = sum_j 2^(s_ij - m_i) vs_j V_j / sum_j 2^(s_ij - m_i)
//
// A sequence's keys are its context, which every drafted token sees, and its
// drafted tokens, of which token i sees those whose bit is set in its mask
// row (without a mask: those up to itself).  The G = Hq / Hk query heads that
// share a key head and a sequence's drafted tokens form the rows of one
// product: a cached byte is read once for each block of rows, of 8 or 16 in
// k_tree_rows, 128 or 256 in k_tree_tile.
//
// Work split.  A segment is one sequence, one key head and one block of rows;
// its keys form tiles of kTile.  All segments' tiles lie on one line, and CTA
// w of W takes the w-th equal part of it, whatever the sequences' lengths: a
// part that covers a segment wholly writes its rows' result, and the others
// leave (m, l, O) in the workspace for k_tree_join, which adds them in tile
// order (no atomics: the same inputs give the same bits).  Lengths are read
// on the device, so a captured call follows them.
#pragma once

#include <cuda.h>  // CUtensorMap (type only; the maps are encoded on the host)

#include "gemm_norm.cuh"  // mbarrier wrappers
#include "kv.cuh"

namespace rarn {
namespace tree {

using kv::Cache;
using kv::Heads;

constexpr int kTile = 64;        // keys of a tile
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCtas = 608;    // parts of the line of tiles, at most
constexpr int kStep = 16;        // keys a warp takes at a time
constexpr unsigned int kWatchTree = 32u;  // watchdog bit: a wait ran out
constexpr unsigned long long kWaitLimitNs = 2000000000ull;

// A segment's parts, for k_tree_join.
struct Join {
    int first, last;  // CTAs whose parts add up to it (last < 0: nothing to add)
    int row0, n;      // its sequence's first drafted token, and how many
    int head, block, pad[2];
};

struct Params {
    Heads q, out;
    Cache cache;
    const int32_t *table;    // [B, width]
    int64_t table_stride;
    int table_width;
    const int32_t *context;  // [B]: cached tokens before the drafted ones
    const int32_t *starts;   // [B + 1]: first drafted token of each sequence
    const uint32_t *mask;    // [tokens, words] or nullptr
    int words;
    int B;
    int64_t tokens;
    int D;
    int G;                   // query heads per key head
    bool bf16;               // type of q and out (else binary16)
    bool out_aligned;        // out's rows on 8-byte boundaries
    float scale_log2;        // scale * log2(e)
    bool whole_steps;        // a step of 16 keys lies inside one page, its scales adjacent on a
                             // 16-byte boundary
    int page_shift;          // log2 of the page size, or -1
    int box;                 // slots of k_tree_tile's TMA boxes

    __device__ __forceinline__ int page_of(int j) const {
        return page_shift >= 0 ? j >> page_shift : j / cache.page_size;
    }
    __device__ __forceinline__ int offset_in_page(int j) const {
        return page_shift >= 0 ? j & (cache.page_size - 1) : j % cache.page_size;
    }
    // workspace
    Join *joins;             // [segments]
    int *count;              // segments of this call
    int max_segs;            // room in joins
    float2 *ml;              // [2 W][rows]
    float *part;             // [2 W][rows][D]
    unsigned int *watchdog;
    unsigned long long wait_limit_ns;
    int stall_fill;          // test hook: in CTA 0 this fill (of its first warp that copies) never
                             // completes (-1: off)
};

// One sequence's share of the line of tiles.
struct Seq {
    int n;       // drafted tokens
    int ctx;     // context length
    int len;     // visible keys at most: ctx + n, as far as the table reaches
    int blocks;  // row blocks
    int tiles;   // tiles of a segment
};

__device__ __forceinline__ Seq seq_of(const Params &p, int b, int rows, int tile) {
    Seq s;
    const int64_t a = p.starts[b], e = p.starts[b + 1];
    s.n = (a >= 0 && e > a && e <= p.tokens) ? static_cast<int>(e - a) : 0;
    const int c = p.context[b];
    s.ctx = c > 0 ? c : 0;
    const int64_t reach = (int64_t)p.table_width * p.cache.page_size;
    const int64_t len = (int64_t)s.ctx + s.n;
    s.len = static_cast<int>(len < reach ? len : reach);
    s.blocks = (int)(((int64_t)s.n * p.G + rows - 1) / rows);
    s.tiles = s.len > 0 ? (s.len + tile - 1) / tile : 1;
    return s;
}

// A segment takes some units of the line for its beginning and end (queries
// read, state joined and written), then one for each of its tiles.  Without
// them a CTA with many short segments worked on when the others were done.
// k_tree_rows, tiles of 64 keys: 64 ragged decode sequences took 129 us with 0
// units, 110 with 2, 106 with 3, 107 with 4, 109 with 6, 111 with 8, 16 short
// ones of few tokens 45 with 4, 52 with 3.  k_tree_tile, tiles of 128: 16 ragged
// sequences of 48 and of 96 rows 63 and 70 us with 4, 59 and 60 with 6, 60 and
// 60 with 8; of 256 rows 135 with 3, 123 with 4 and 6, 128 with 8.
__device__ __forceinline__ constexpr int begin_units(int tile) { return tile == kTile ? 4 : 6; }

__device__ __forceinline__ int64_t units_of(const Params &p, const Seq &s, int tile) {
    return (int64_t)p.cache.heads * s.blocks * (s.tiles + begin_units(tile));
}

// Where a CTA's part of the line begins: CTA w has `each` tiles, one more
// while w < `more`.
struct Cursor {
    int total;         // tiles on the line
    int parts;         // CTAs with a part
    int each, more;
    int lo, hi;        // this CTA's part
    int b;             // sequence of lo
    int base;          // first tile of that sequence on the line
    int seg0;          // segments before that sequence
};

// Prefix sums over the sequences by the whole CTA: thread i takes the i-th
// run of consecutive ones.  `sh` holds kN / 16 + 3 words.
template <int kN>
__device__ __forceinline__ Cursor find_part(const Params &p, int rows, int tile, int64_t *sh) {
    const int run = (p.B + kN - 1) / kN;
    const int b0 = threadIdx.x * run, b1 = min(b0 + run, p.B);
    int64_t mine = 0, segs = 0;
    if (threadIdx.x < kN)
        for (int b = b0; b < b1; ++b) {
            const Seq s = seq_of(p, b, rows, tile);
            mine += units_of(p, s, tile);
            segs += (int64_t)p.cache.heads * s.blocks;
        }
    // inclusive scans inside the warp, then over the warps
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t u = mine, g = segs;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, u, d);
        const int64_t y = __shfl_up_sync(0xffffffffu, g, d);
        if (lane >= d) {
            u += x;
            g += y;
        }
    }
    constexpr int kW = kN / 32;
    if (warp < kW && lane == 31) {
        sh[warp] = u;
        sh[kW + warp] = g;
    }
    __syncthreads();
    int64_t before = 0, total = 0, gbefore = 0, gtotal = 0;
#pragma unroll
    for (int i = 0; i < kW; ++i) {
        if (i < warp) {
            before += sh[i];
            gbefore += sh[kW + i];
        }
        total += sh[i];
        gtotal += sh[kW + i];
    }
    // starts that do not rise name more rows than there are: nothing is done
    const bool sound = gtotal <= p.max_segs && total < (int64_t(1) << 31);
    if (!sound) total = 0;
    Cursor c;
    c.total = (int)total;
    c.parts = total < gridDim.x ? (int)total : (int)gridDim.x;
    c.each = c.parts ? (unsigned)c.total / (unsigned)c.parts : 0;
    c.more = c.total - c.each * c.parts;
    const int w = blockIdx.x;
    c.lo = w < c.parts ? w * c.each + min(w, c.more) : c.total;
    c.hi = w < c.parts ? c.lo + c.each + (w < c.more ? 1 : 0) : c.total;
    if (w == 0 && threadIdx.x == 0) {
        *p.count = sound ? (int)gtotal : 0;
        if (!sound) atomicOr(p.watchdog, kv::kWatchIndex);
    }
    const int64_t first = before + u - mine;
    if (threadIdx.x < kN && c.lo < c.hi && c.lo >= first && c.lo < first + mine) {
        int64_t at = first, seg = gbefore + g - segs;
        int b = b0;
        for (;; ++b) {
            const Seq s = seq_of(p, b, rows, tile);
            const int64_t n = units_of(p, s, tile);
            if (c.lo < at + n) break;
            at += n;
            seg += (int64_t)p.cache.heads * s.blocks;
        }
        sh[2 * kW] = b;
        sh[2 * kW + 1] = at;
        sh[2 * kW + 2] = seg;
    }
    __syncthreads();
    c.b = c.lo < c.hi ? (int)sh[2 * kW] : 0;
    c.base = (int)sh[2 * kW + 1];
    c.seg0 = (int)sh[2 * kW + 2];
    return c;
}

// The CTA whose part holds tile `t` of the line (Cursor's each and more).
__device__ __forceinline__ int part_of(int each, int more, int t) {
    const int edge = more * (each + 1);
    return t < edge ? (unsigned)t / (unsigned)(each + 1)
                    : more + (unsigned)(t - edge) / (unsigned)each;
}

// A key's place in the cache: code and scale offsets of (its page, its slot),
// head included; code < 0: no such page.
struct KeyAt {
    int64_t code, scale;
};

__device__ __forceinline__ KeyAt place(const Params &p, int64_t page, int at, int head) {
    KeyAt k;
    k.code = page * p.cache.page_stride + (int64_t)head * p.cache.head_stride +
             at * p.cache.slot_stride;
    k.scale = page * p.cache.s_page + (int64_t)head * p.cache.s_head + at * p.cache.s_slot;
    return k;
}

// Whether drafted token `i` (of its sequence) sees drafted token `d`; `row` is
// its row of the mask.
__device__ __forceinline__ bool sees(const Params &p, int64_t row, int i, int d) {
    if (!p.mask) return d <= i;
    return d < p.words * 32 && ((p.mask[row * p.words + (d >> 5)] >> (d & 31)) & 1u);
}

__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
    return DT<__half>::f2w(a, b);
}

// S += K Q^T: 16 keys of 32 codes by 8 rows of 32 e4m3 pieces.
template <bool kE5M2>
__device__ __forceinline__ void mma_codes(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (kE5M2) {
        asm volatile(
            "mma.sync.aligned.m16n8k32.row.col.f32.e5m2.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    } else {
        asm volatile(
            "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
}

// The first of a chain: S = K Q^T.
template <bool kE5M2>
__device__ __forceinline__ void mma_codes_first(float (&d)[4], uint32_t a0, uint32_t a1,
                                                uint32_t a2, uint32_t a3, uint32_t b0,
                                                uint32_t b1) {
    if constexpr (kE5M2) {
        asm volatile(
            "mma.sync.aligned.m16n8k32.row.col.f32.e5m2.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    } else {
        asm volatile(
            "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    }
}

// O += V^T P: 16 elements by 8 rows over 16 keys, binary16.
__device__ __forceinline__ void mma_half(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Asynchronous copies of 16 and 4 bytes; zeros where `live` is false (nothing
// is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(live ? 4 : 0)
                 : "memory");
}

__device__ __forceinline__ void copies_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A box of codes: bytes x .., slots y .. of one head and page.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x,
                                        int y, int head, int page) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(head), "r"(page)
        : "memory");
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// Bounded wait: false, with the watchdog bit set, when it runs out.
__device__ __forceinline__ bool wait_stage(const Params &p, uint32_t bar, uint32_t parity) {
    if (gemm::mbar_try_wait(bar, parity)) return true;
    unsigned long long t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (gemm::mbar_try_wait(bar, parity)) return true;
        if ((i & 127u) == 0) {
            const unsigned long long t = gemm::now_ns();
            if (t0 == 0) {
                t0 = t;
            } else if (t - t0 > p.wait_limit_ns) {
                atomicOr(p.watchdog, kWatchTree);
                return false;
            }
        }
    }
}

__device__ __forceinline__ void lds(uint32_t (&w)[4], uint32_t a) {
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(a)
                 : "memory");
}

__device__ __forceinline__ void lds(uint32_t (&w)[2], uint32_t a) {
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
}

__device__ __forceinline__ void lds(uint32_t (&w)[1], uint32_t a) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(a) : "memory");
}

__device__ __forceinline__ float lds_f(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// One step of a warp in shared memory: kStep keys' codes and their values'
// codes, rows in halves of at most 128 bytes; apart from them (kTail) the
// scales of both and a word whose bit j says that key j exists.  A row's
// 16-byte chunks are stored at their index xor a few bits of the row, which is
// the TMA swizzle of 128- and 64-byte rows: the lanes of one load, which read
// one or two chunks of several rows, meet different banks.
template <int D>
struct StepLayout {
    static constexpr int kHalf = D % 128 == 0 ? 128 : D;  // bytes of a row kept together
    static constexpr int kChunks = kHalf / 16;
    static constexpr int kLow = kChunks & -kChunks;
    static constexpr int kXor = (kLow < 8 ? kLow : 8) - 1;
    // rows of 64 bytes: two share a line of banks
    static constexpr int kShift = kHalf < 128 ? 1 : 0;
    static constexpr int kV = kStep * D, kBytes = 2 * kStep * D;
    static constexpr int kScaleV = 4 * kStep, kOk = 8 * kStep, kTail = kOk + 16;
    __device__ __forceinline__ static int chunk(int row, int x) {
        const int half = x / kChunks, y = x % kChunks;
        return half * (kStep * kHalf) + row * kHalf + ((y ^ ((row >> kShift) & kXor)) << 4);
    }
};

// A stage of a warp's ring: where its codes and its tail are.
struct Stage {
    uint32_t codes, tail;
};

// N words at byte `at` of row `row` (a multiple of 4 N, or of 16): as wide as
// they stay inside a chunk.
template <int D, int N>
__device__ __forceinline__ void load_row(uint32_t (&w)[N], uint32_t base, int row, int at) {
    constexpr int W = N % 4 == 0 ? 4 : N % 2 == 0 ? 2 : 1;
#pragma unroll
    for (int i = 0; i < N; i += W) {
        const int byte = at + 4 * i;
        uint32_t t[W];
        lds(t, base + StepLayout<D>::chunk(row, byte >> 4) + (byte & 15));
#pragma unroll
        for (int j = 0; j < W; ++j) w[i + j] = t[j];
    }
}

// Slack of the running maximum, in powers of two: a row's weights may reach
// 2^kSlack before its sums are rescaled, so that a rescale (a reduction over
// the warp and a pass over the accumulators) is rare.
constexpr float kSlack = 3.f;
// Weights enter the second product in binary16 as p vs by, `by` the power of
// two that brings the row's largest |vs| to [2^11, 2^12), so at most 2^15: what
// falls under 2^-24 of that, 2^-35 of the largest term, is lost, which 2^19
// keys cannot add up to a rounding of the result.  A row's `by` goes by the
// keys that it sees.  The divisor sums the weights before that rounding (64
// decode sequences 107 -> 103 us against taking each weight's rounding into
// it).
constexpr int kWeightBits = 12;
constexpr int kMostBy = 127 + 112;  // exponent field of `by` before any key

__device__ __forceinline__ float from_exponent(int field) { return __int_as_float(field << 23); }
__device__ __forceinline__ int exponent_of(float x) { return __float_as_int(x) >> 23; }

// The exponent field of `by` for a largest |vs| (0: none yet).
__device__ __forceinline__ int by_for(float most) {
    return min(kMostBy, 127 + kWeightBits - (exponent_of(most) - 126));
}

// A maximum before any score: finite, so that a hidden key's weight is 0.
constexpr float kNoScore = -3e38f;

// A warp's running softmax and accumulators.
template <int D, int NQ>
struct RowState {
    float m[NQ][2];    // running maximum of the lane's rows (log2 units), kNoScore: none yet
    float l[NQ][2];    // this lane's keys' sum of weights
    float by[NQ][2];   // what weights are multiplied with
    float ref;         // the least 2^kWeightBits / by of the lane's rows
    float o[D / 16][NQ][4];

    __device__ __forceinline__ void clear() {
        ref = from_exponent(254 + kWeightBits - kMostBy);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            by[n][0] = by[n][1] = from_exponent(kMostBy);
            m[n][0] = m[n][1] = kNoScore;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int t = 0; t < D / 16; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[t][n][i] = 0.f;
        }
    }
};

// Largest value of v over the lanes that share c (rows 2c, 2c + 1).
__device__ __forceinline__ float max_over_keys(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}

__device__ __forceinline__ float sum_over_keys(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 4);
    v += __shfl_xor_sync(0xffffffffu, v, 8);
    return v + __shfl_xor_sync(0xffffffffu, v, 16);
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm volatile("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A CTA's share of one segment.
struct Segment {
    int b, head, block;
    Seq s;
    int64_t row0;  // first drafted token of the sequence
};

// Row r of a segment's block: token, query head; false past the last row.
__device__ __forceinline__ bool row_of(const Params &p, const Segment &sg, int rows, int r, int &i,
                                       int &h) {
    const int R = sg.block * rows + r;
    i = R / p.G;
    h = sg.head * p.G + (R - i * p.G);
    return i < sg.s.n;
}

// Whether one of four codes is NaN or infinite.
template <bool kE5M2>
__device__ __forceinline__ bool any_nonfinite(uint32_t w) {
    // e4m3: magnitude 0x7f; e5m2: exponent field 31
    constexpr uint32_t top = kE5M2 ? 0x7c7c7c7cu : 0x7f7f7f7fu;
    return __vcmpeq4(w & top, top) != 0;
}

// A warp's copies of the step of keys j0 .. into a stage of its ring, as
// 16-byte asynchronous copies: any layout of the cache.
template <int D>
__device__ __forceinline__ void issue_step(const Params &p, const Segment &sg, const Stage &stage,
                                           int j0) {
    using L = StepLayout<D>;
    const int lane = threadIdx.x & 31;
    // lane r (and r + 16) finds key r's place; the others take it by shuffle
    const int j = j0 + (lane & 15);
    KeyAt mine{-1, 0};
    if (j < sg.s.len) {
        const int pg = p.page_of(j);
        const int64_t page = p.table[sg.b * p.table_stride + pg];
        if (page >= 0 && page < p.cache.pages)
            mine = place(p, page, j - pg * p.cache.page_size, sg.head);
        else
            atomicOr(p.watchdog, kv::kWatchIndex);
    }
    const uint32_t ok = __ballot_sync(0xffffffffu, mine.code >= 0) & 0xffffu;
    const float *sc = lane < 16 ? p.cache.k_scale : p.cache.v_scale;
    copy4(stage.tail + 4 * lane, sc + mine.scale, mine.code >= 0);
    constexpr int kRowChunks = D / 16;
#pragma unroll
    for (int x0 = 0; x0 < kStep * kRowChunks; x0 += 32) {
        const int x = x0 + lane;
        const bool in = x < kStep * kRowChunks;
        const int row = in ? x / kRowChunks : 0, ch = x % kRowChunks;
        const int64_t at = __shfl_sync(0xffffffffu, mine.code, row);
        if (in) {
            const uint32_t dst = stage.codes + L::chunk(row, ch);
            copy16(dst, p.cache.k + (at >= 0 ? at + ch * 16 : 0), at >= 0);
            copy16(dst + L::kV, p.cache.v + (at >= 0 ? at + ch * 16 : 0), at >= 0);
        }
    }
    if (lane == 0)
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(stage.tail + L::kOk), "r"(ok) : "memory");
}

// The same by TMA, from one lane, where a step lies inside one page and its
// scales are adjacent: the box of its keys' rows and that of its values', and
// the two runs of scales.  `page` is the page's number, loaded ahead.  Slots
// behind the sequence's end come along and are masked.  `extra`: bytes that are
// awaited and never come (the test hook).  64 sequences of up to
// 8192 tokens, 8 key heads of 128, one token each: 125.5 us, with the copies
// above 131.7 (both before segments' ends counted in the split).
template <int D>
__device__ __forceinline__ void issue_step_tma(const Params &p, const Segment &sg,
                                               const CUtensorMap *kmap, const CUtensorMap *vmap,
                                               const Stage &stage, uint32_t bar, int j0,
                                               int page, uint32_t extra) {
    using L = StepLayout<D>;
    const bool have = page >= 0 && page < p.cache.pages;
    const int live = min(kStep, sg.s.len - j0);
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(stage.tail + L::kOk),
                 "r"(have ? 0xffffu >> (kStep - live) : 0u)
                 : "memory");
    if (!have) {
        atomicOr(p.watchdog, kv::kWatchIndex);
        gemm::mbar_arrive(bar);
        return;
    }
    const int at = p.offset_in_page(j0);
    const bool rows = p.cache.mode == Q_ROW;
    gemm::mbar_arrive_expect_tx(bar, L::kBytes + (rows ? 8 * kStep : 0) + extra);
#pragma unroll
    for (int h = 0; h < D / L::kHalf; ++h) {
        const uint32_t dst = stage.codes + h * (kStep * L::kHalf);
        tma_box(dst, kmap, bar, h * L::kHalf, at, sg.head, page);
        tma_box(dst + L::kV, vmap, bar, h * L::kHalf, at, sg.head, page);
    }
    if (rows) {
        const int64_t sc = page * p.cache.s_page + sg.head * p.cache.s_head + at;
        bulk_copy(stage.tail, p.cache.k_scale + sc, 4 * kStep, bar);
        bulk_copy(stage.tail + L::kScaleV, p.cache.v_scale + sc, 4 * kStep, bar);
    }
}

// One step: scores, softmax, second product.
template <int D, int NQ, int NP, bool kE5M2>
__device__ __forceinline__ void consume_step(const Params &p, const Segment &sg, const Stage &stage,
                                             int j0, const uint32_t (&q)[D / 32][NP][NQ][2],
                                             const float (&cs)[NQ][2],
                                             const int (&tok)[NQ][2], RowState<D, NQ> &rs) {
    using L = StepLayout<D>;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    float s[NQ][4];
    {
        // the pieces of q are 2^-4 apart: one accumulator each
        float t[NP][NQ][4];
        uint32_t k0[D / 16], k1[D / 16];
        load_row<D>(k0, stage.codes, g, c * (D / 4));
        load_row<D>(k1, stage.codes, g + 8, c * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int u = 0; u < NP; ++u)
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    if (i == 0)
                        mma_codes_first<kE5M2>(t[u][n], k0[0], k1[0], k0[1], k1[1],
                                               q[0][u][n][0], q[0][u][n][1]);
                    else
                        mma_codes<kE5M2>(t[u][n], k0[2 * i], k1[2 * i], k0[2 * i + 1],
                                         k1[2 * i + 1], q[i][u][n][0], q[i][u][n][1]);
                }
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[n][i] = t[NP - 1][n][i];
#pragma unroll
                for (int u = NP - 2; u >= 0; --u) s[n][i] = fmaf(s[n][i], 0.0625f, t[u][n][i]);
            }
    }
    float ks0, ks1, vs0, vs1;
    if (p.cache.mode == Q_ROW) {
        ks0 = lds_f(stage.tail + 4 * g);
        ks1 = lds_f(stage.tail + 4 * g + 32);
        vs0 = lds_f(stage.tail + L::kScaleV + 4 * g);
        vs1 = lds_f(stage.tail + L::kScaleV + 4 * g + 32);
    } else {
        ks0 = ks1 = __ldg(p.cache.k_scale);
        vs0 = vs1 = __ldg(p.cache.v_scale);
    }
    uint32_t ok[1];
    lds(ok, stage.tail + L::kOk);
    // s[n][0..1]: key g, rows 2c, 2c + 1; s[n][2..3]: key g + 8
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][i] *= (i < 2 ? ks0 : ks1) * cs[n][i & 1];
    const bool edge = ok[0] != 0xffffu || j0 + kStep > sg.s.ctx;  // uniform
    uint32_t hidden = 0;  // bit 4 n + i: s[n][i] is not visible
    if (__builtin_expect(edge, 0)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = g + 8 * h, d = j0 + j - sg.s.ctx;
            const bool exists = (ok[0] >> j) & 1u;
            if (!exists) (h ? vs1 : vs0) = 0.f;
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = tok[n][e];
                    const bool vis = exists && i >= 0 && (d < 0 || sees(p, sg.row0 + i, i, d));
                    if (!vis) {
                        hidden |= 1u << (4 * n + 2 * h + e);
                        s[n][2 * h + e] = -INFINITY;
                    }
                }
        }
    }
    bool grow = !(fabsf(vs0) <= rs.ref) || !(fabsf(vs1) <= rs.ref);
    float top[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        top[n][0] = fmaxf(s[n][0], s[n][2]);
        top[n][1] = fmaxf(s[n][1], s[n][3]);
        grow |= top[n][0] > rs.m[n][0] + kSlack || top[n][1] > rs.m[n][1] + kSlack;
    }
    if (__any_sync(0xffffffffu, grow)) {
        // of finite value scales the largest that a row sees
        const float v0 = fabsf(vs0) < INFINITY ? fabsf(vs0) : 0.f,
                    v1 = fabsf(vs1) < INFINITY ? fabsf(vs1) : 0.f;
        int least = 0;
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t hid = hidden >> (4 * n + e);
                const float vm =
                    max_over_keys(fmaxf(hid & 1u ? 0.f : v0, hid & 4u ? 0.f : v1));
                const int was = exponent_of(rs.by[n][e]), is = min(was, by_for(vm));
                const float rr = is - was < -126 ? 0.f : from_exponent(127 + is - was);
                rs.by[n][e] = from_exponent(is);
                least = max(least, is);
                const float m = fmaxf(rs.m[n][e], max_over_keys(top[n][e]));
                const float a = rs.m[n][e] == m ? 1.f : exp2_fast(rs.m[n][e] - m);
                rs.m[n][e] = m;
                rs.l[n][e] *= a;
#pragma unroll
                for (int t = 0; t < D / 16; ++t) {
                    rs.o[t][n][e] *= a * rr;
                    rs.o[t][n][2 + e] *= a * rr;
                }
            }
        rs.ref = from_exponent(254 + kWeightBits - least);
    }
    uint32_t pb[NQ][2];
    float x[NQ][4];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        float pr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            pr[i] = exp2_fast(s[n][i] - rs.m[n][i & 1]);
            x[n][i] = pr[i] * ((i < 2 ? vs0 : vs1) * rs.by[n][i & 1]);
        }
        if (__builtin_expect(edge, 0)) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if ((hidden >> (4 * n + i)) & 1u) x[n][i] = 0.f;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t packed = pack_h2(x[n][2 * h], x[n][2 * h + 1]);
            pb[n][h] = transpose_8x8(packed);
            rs.l[n][0] += pr[2 * h];
            rs.l[n][1] += pr[2 * h + 1];
        }
    }
    // values of keys 2c, 2c + 1, 2c + 8, 2c + 9, this lane's eighth of the row
    uint32_t v[4][D / 32];
#pragma unroll
    for (int h = 0; h < 4; ++h)
        load_row<D>(v[h], stage.codes + L::kV, 2 * c + (h & 1) + (h >> 1) * 8, g * (D / 8));
    if (__builtin_expect(edge, 0)) {
        // Values that are NaN or infinite and not visible to every row: in the
        // product 0 times such a value would be NaN, so those keys leave it
        // (their codes become zero) and are added to the rows that see them.
        uint32_t bad = 0;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            bool any = false;
            const bool exists = (ok[0] >> (2 * c + (h & 1) + (h >> 1) * 8)) & 1u;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                if (!exists) v[h][i] = 0;  // what a slot behind the end holds
                any |= any_nonfinite<kE5M2>(v[h][i]);
            }
            if (any) bad |= 1u << (2 * c + (h & 1) + (h >> 1) * 8);
        }
        bad = __reduce_or_sync(0xffffffffu, bad);
        if (bad) {
#pragma unroll 1
            for (int j = 0; j < kStep; ++j) {
                if (!((bad >> j) & 1u)) continue;
                const int from = 4 * (j & 7) + c;
                const uint32_t hid = __shfl_sync(0xffffffffu, hidden, from);
                uint32_t w[D / 32];
                load_row<D>(w, stage.codes + L::kV, j, g * (D / 8));
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float wt =
                            __shfl_sync(0xffffffffu, j < 8 ? x[n][e] : x[n][2 + e], from);
                        if (!((hid >> (4 * n + (j < 8 ? e : 2 + e))) & 1u)) {
#pragma unroll
                            for (int t = 0; t < D / 16; ++t) {
                                const uint32_t two = t & 1 ? w[t / 2] >> 16 : w[t / 2] & 0xffffu;
                                const float2 f = DT<__half>::w2f(kv::codes2_to_h2<kE5M2>(two));
                                rs.o[t][n][e] += wt * f.x;
                                rs.o[t][n][2 + e] += wt * f.y;
                            }
                        }
                    }
            }
#pragma unroll
            for (int h = 0; h < 4; ++h)
                if ((bad >> (2 * c + (h & 1) + (h >> 1) * 8)) & 1u) {
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) v[h][i] = 0;
                }
        }
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        // bytes of two keys interleaved: two elements per 32-bit word
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t lo = __byte_perm(v[0][i], v[1][i], u ? 0x7362 : 0x5140);
            const uint32_t hi = __byte_perm(v[2][i], v[3][i], u ? 0x7362 : 0x5140);
            uint32_t a0, a1, a2, a3;
            kv::codes4_to_h2<kE5M2>(lo, a0, a1);
            kv::codes4_to_h2<kE5M2>(hi, a2, a3);
#pragma unroll
            for (int n = 0; n < NQ; ++n)
                mma_half(rs.o[2 * i + u][n], a0, a1, a2, a3, pb[n][0], pb[n][1]);
        }
    }
}

__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }

// The block's query rows as the second operand of S = K Q^T.  Each row is
// scaled by a power of two that brings its largest magnitude to [128, 256),
// then split into NP e4m3 pieces, piece u the rounded rest times 2^4u: two
// pieces hold a bfloat16's 8 bits and three a binary16's 11 exactly, down to
// 2^-22 of the row's largest.  The keys' codes thus enter the matrix unit as
// they are, at its 8-bit rate.  cs: what undoes the scaling, times the softmax
// scale, and tok: the token (-1: none), for the lane's rows 2c, 2c + 1.
template <int D, int NQ, int NP>
__device__ __forceinline__ void load_queries(const Params &p, const Segment &sg,
                                             uint32_t (&q)[D / 32][NP][NQ][2],
                                             float (&cs)[NQ][2], int (&tok)[NQ][2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        int i, h;
        const bool live = row_of(p, sg, 8 * NQ, 8 * n + g, i, h);
        float f[D / 4];
        float amax = 0.f;
        bool finite = true;
        const int64_t at = (sg.row0 + i) * p.q.ts + (int64_t)h * p.q.hs + c * (D / 4);
#pragma unroll
        for (int e = 0; e < D / 4; e += 8) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (live) w = ld_stream(static_cast<const uint16_t *>(p.q.data) + at + e);
            float x[8];
            if (NP == 2) DT<__nv_bfloat16>::unpack(w, x);
            else DT<__half>::unpack(w, x);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                f[e + u] = x[u];
                amax = fmaxf(amax, fabsf(x[u]));
                finite = finite && fabsf(x[u]) < INFINITY;
            }
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        int ex = amax > 0.f && amax < INFINITY ? (int)(__float_as_uint(amax) >> 23) - 127 : 7;
        ex = max(ex, -100);
        const float by = power_of_two(7 - ex), back = power_of_two(ex - 7) * p.scale_log2;
#pragma unroll
        for (int s = 0; s < D / 32; ++s)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float r[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) r[e] = f[8 * s + 4 * half + e] * by;
#pragma unroll
                for (int u = 0; u < NP; ++u) {
                    const uint32_t lo = fp8x2(r[0], r[1], Q_E4M3), hi = fp8x2(r[2], r[3], Q_E4M3);
                    q[s][u][n][half] = finite ? lo | (hi << 16) : 0x7f7f7f7fu;
                    const float2 a = kv::codes2_to_f2(lo, Q_E4M3), b = kv::codes2_to_f2(hi, Q_E4M3);
                    r[0] = (r[0] - a.x) * 16.f;
                    r[1] = (r[1] - a.y) * 16.f;
                    r[2] = (r[2] - b.x) * 16.f;
                    r[3] = (r[3] - b.y) * 16.f;
                }
            }
        cs[n][0] = __shfl_sync(0xffffffffu, back, 8 * c);
        cs[n][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
        const int token = live ? i : -1;
        tok[n][0] = __shfl_sync(0xffffffffu, token, 8 * c);
        tok[n][1] = __shfl_sync(0xffffffffu, token, 8 * c + 4);
    }
}

// Four adjacent elements of a result row, rounded to its type.
__device__ __forceinline__ void store_out4(const Params &p, int64_t token, int h, int d,
                                           const float4 &v) {
    const int64_t at = token * p.out.ts + (int64_t)h * p.out.hs + d;
    uint2 w;
    if (p.bf16) w = make_uint2(DT<__nv_bfloat16>::f2w(v.x, v.y), DT<__nv_bfloat16>::f2w(v.z, v.w));
    else w = make_uint2(DT<__half>::f2w(v.x, v.y), DT<__half>::f2w(v.z, v.w));
    uint16_t *dst = static_cast<uint16_t *>(p.out.data) + at;
    if (p.out_aligned) {
        *reinterpret_cast<uint2 *>(dst) = w;
    } else {
        dst[0] = (uint16_t)w.x;
        dst[1] = (uint16_t)(w.x >> 16);
        dst[2] = (uint16_t)w.y;
        dst[3] = (uint16_t)(w.y >> 16);
    }
}

// Shared memory of a CTA: each warp's ring of kStages steps, over which the
// join of the warps is laid at a segment's end, then the steps' tails.
template <int D, int NQ, int kStages>
struct Smem {
    static constexpr int kRing = kWarps * kStages * StepLayout<D>::kBytes;
    static constexpr int kPad = D + 4;  // floats per row of the join
    static constexpr int kJoin = kWarps * 8 * NQ * kPad * 4;
    static constexpr int kTails = kRing > kJoin ? kRing : kJoin;
    static constexpr int kBytes = kTails + kWarps * kStages * StepLayout<D>::kTail + 1024;
};

// Four warps share a segment's tiles, kStep keys each in turn, with their own
// copies in flight and their own running maxima and sums, so nothing in the
// loop waits for another warp; they are joined through shared memory at the
// end of the CTA's share of the segment.
//
// Bound by memory where sequences are long: 64 of up to 8192 tokens, 8 key
// heads of 128, one token of 32 heads each, take 101 us with the join (5.4 TB/s,
// 80 % of a copy's rate); there 60 % of all issue slots and half the ALU's are
// taken, by the values' conversion above all, and the ends of 512 segments come
// on top.  One sequence's token takes 12 us, two launches and the chain of
// lengths, page, keys and parts.  mma.sync serves up to 16 rows, whose products
// take less than their keys' reading.
template <int D, int NQ, int NP, bool kE5M2, int kStages, bool kTma>
__global__ void __launch_bounds__(kThreads, NQ == 1 && D <= 128 ? 4 : 2)
    k_tree_rows(const Params p, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
    using S = Smem<D, NQ, kStages>;
    using L = StepLayout<D>;
    constexpr int kRows = 8 * NQ;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int64_t sh_part[16];
    __shared__ float sh_m[kWarps][kRows], sh_l[kWarps][kRows];
    __shared__ __align__(8) uint64_t sh_bar[kWarps][kStages];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    float *sh_o = reinterpret_cast<float *>(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * kStages * L::kBytes;
    const uint32_t tails = smem_u32(smem) + S::kTails + warp * kStages * L::kTail;
    const uint32_t bars = smem_u32(&sh_bar[warp][0]);
    auto stage_at = [&](int i) { return Stage{ring + i * L::kBytes, tails + i * L::kTail}; };
    if (kTma) {
        if (lane == 0)
            for (int i = 0; i < kStages; ++i) gemm::mbar_init(bars + 8 * i, 1);
        gemm::fence_async_shared();
        __syncwarp();
    }
    uint32_t phases = 0;  // bit i: parity of stage i's next fill
    bool sound = true;    // no wait has run out
    int to_stall = blockIdx.x == 0 && warp == 0 ? p.stall_fill : -1;  // fills until that one
    grid_dependency_wait();
    grid_launch_dependents();
    const Cursor cur = find_part<kThreads>(p, kRows, kTile, sh_part);
    int at = cur.lo, base = cur.base, seg0 = cur.seg0;
    Segment sg;
    sg.b = cur.b;
    while (at < cur.hi) {
        sg.s = seq_of(p, sg.b, kRows, kTile);
        constexpr int kBegin = begin_units(kTile);
        const int units = (int)units_of(p, sg.s, kTile);
        if (at >= base + units) {
            base += units;
            seg0 += p.cache.heads * sg.s.blocks;
            ++sg.b;
            continue;
        }
        const int each = sg.s.tiles + kBegin;
        const int which = (unsigned)(at - base) / (unsigned)each;
        const int x0 = at - base - which * each, x1 = min(x0 + cur.hi - at, each);
        at += x1 - x0;
        const int t0 = max(x0 - kBegin, 0), t1 = x1 - kBegin;
        if (t1 <= t0) continue;
        sg.head = (unsigned)which / (unsigned)sg.s.blocks;
        sg.block = which - sg.head * sg.s.blocks;
        sg.row0 = p.starts[sg.b];

        const int j1 = min(t1 * kTile, sg.s.len);
        const int first = sound ? t0 * kTile + warp * kStep : j1;
        const int32_t *pages = p.table + sg.b * p.table_stride;
        // the page of the step that is copied next, loaded a step ahead
        int page = kTma && first < j1 ? pages[p.page_of(first)] : 0;
        int ahead = first;  // step that is copied next
        auto issue = [&](int i) {
            if (kTma) {
                if (ahead < j1) {
                    const int now = page, nx = ahead + kTile;
                    if (nx < j1) page = pages[p.page_of(nx)];
                    if (lane == 0)
                        issue_step_tma<D>(p, sg, &kmap, &vmap, stage_at(i), bars + 8 * i, ahead,
                                          now, to_stall == 0 ? 16u : 0u);
                    --to_stall;
                }
            } else {
                if (ahead < j1) issue_step<D>(p, sg, stage_at(i), ahead);
                copies_commit();
            }
            ahead += kTile;
        };
#pragma unroll 1
        for (int i = 0; i < kStages - 1; ++i) issue(i);
        uint32_t q[D / 32][NP][NQ][2];
        float cs[NQ][2];
        int tok[NQ][2];
        load_queries<D, NQ, NP>(p, sg, q, cs, tok);
        RowState<D, NQ> rs;
        rs.clear();
        int stage = 0;
#pragma unroll 1
        for (int j = first; j < j1; j += kTile) {
            if (kTma) {
                const bool here = wait_stage(p, bars + 8 * stage, (phases >> stage) & 1u);
                phases ^= 1u << stage;
                sound = __all_sync(0xffffffffu, here);
                if (!sound) {
                    // take no more steps, and leave no copy in flight
                    const int left = min((j1 - j + kTile - 1) / kTile, kStages - 1);
                    for (int i = 1; i < left; ++i) {
                        const int x = (stage + i) % kStages;
                        wait_stage(p, bars + 8 * x, (phases >> x) & 1u);
                        phases ^= 1u << x;
                    }
                    break;
                }
            } else {
                copies_wait<kStages - 2>();
            }
            __syncwarp();  // every lane's copies of this step; and the next stage is free
            issue(stage == 0 ? kStages - 1 : stage - 1);
            consume_step<D, NQ, NP, kE5M2>(p, sg, stage_at(stage), j, q, cs, tok, rs);
            stage = stage == kStages - 1 ? 0 : stage + 1;
        }
        if (!kTma) copies_wait<0>();
        if (kTma && !sound) {  // what is missing is not passed over
#pragma unroll
            for (int n = 0; n < NQ; ++n) rs.l[n][0] = rs.l[n][1] = NAN;
        }
        // join the warps
        __syncthreads();  // every warp's ring is free
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float l = sum_over_keys(rs.l[n][e]);
                if (g == 0) {
                    sh_m[warp][8 * n + 2 * c + e] =
                        rs.m[n][e] == kNoScore ? -INFINITY : rs.m[n][e];
                    sh_l[warp][8 * n + 2 * c + e] = l;
                }
            }
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const float unit[2] = {from_exponent(254 - exponent_of(rs.by[n][0])),
                                   from_exponent(254 - exponent_of(rs.by[n][1]))};
#pragma unroll
            for (int t = 0; t < D / 16; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sh_o[(warp * kRows + 8 * n + 2 * c + (i & 1)) * S::kPad + g * (D / 8) + 2 * t +
                         (i >> 1)] = rs.o[t][n][i] * unit[i & 1];
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == sg.s.tiles;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (t0 == 0 ? 1 : 0);
        for (int x = threadIdx.x; x < kRows * (D / 4); x += kThreads) {
            const int r = x / (D / 4), d = (x - r * (D / 4)) * 4;
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sh_m[w][r]);
            float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = sh_m[w][r];
                const float f = mw == -INFINITY ? 0.f : mw == m ? 1.f : exp2f(mw - m);
                const float4 o = *reinterpret_cast<const float4 *>(
                    &sh_o[(w * kRows + r) * S::kPad + d]);
                l += f * sh_l[w][r];
                acc[0] += f * o.x;
                acc[1] += f * o.y;
                acc[2] += f * o.z;
                acc[3] += f * o.w;
            }
            if (whole) {
                int i, h;
                if (row_of(p, sg, kRows, r, i, h)) {
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    store_out4(p, sg.row0 + i, h, d,
                               make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv));
                }
            } else {
                if (d == 0) p.ml[slot * kRows + r] = make_float2(m, l);
                *reinterpret_cast<float4 *>(p.part + (slot * kRows + r) * D + d) =
                    make_float4(acc[0], acc[1], acc[2], acc[3]);
            }
        }
        if (t0 == 0 && threadIdx.x == 0)
            p.joins[seg0 + which] =
                Join{(int)blockIdx.x, whole ? -1 : part_of(cur.each, cur.more, at - x1 + each - 1),
                     (int)sg.row0, sg.s.n, sg.head, sg.block, 0, 0};
        gemm::fence_async_shared();  // the join's accesses before the next copies
        __syncthreads();
    }
}

// Adds the parts of the segments that no CTA covered wholly, in tile order.
// kSplit warps share a row's parts: 1 where there are many segments of a few
// parts, 8 where there are few of many (one long sequence: 19 to 76 parts each).
// Bound by instructions rather than by its reads, which come from L2: 128
// segments of 256 rows in two or three parts, 8 us; two parts at a time there
// (four: 10 us).
template <int D, int kSplit>
__global__ void __launch_bounds__(256) k_tree_join(const Params p, int rows) {
    constexpr int N = (D + 127) / 128;
    constexpr int kRows = 8 / kSplit;
    __shared__ float2 sh_ml[8];
    __shared__ __align__(16) float4 sh_o[8][32 * N];
    grid_dependency_wait();
    grid_launch_dependents();
    const int seg = blockIdx.x;
    const Join jn = p.joins[seg];
    if (seg >= *p.count || jn.last < 0) return;  // beyond the count: never written
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.y * kRows + warp / kSplit, sub = warp % kSplit;
    const int R = jn.block * rows + r, i = R / p.G;
    const bool live = i < jn.n;
    if (kSplit == 8 && !live) return;  // the whole CTA: one row
    // the first part is in its CTA's slot 1, the later ones in slot 0
    auto slot = [&](int w) { return (2 * (int64_t)w + (w == jn.first ? 1 : 0)) * rows + r; };
    float m = -INFINITY, l = 0.f;
    float4 acc[N];
#pragma unroll
    for (int n = 0; n < N; ++n) acc[n] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
        constexpr int U = kSplit == 1 ? 2 : 4;
        for (int w0 = jn.first + sub; w0 <= jn.last; w0 += U * kSplit) {
            float2 v[U];
            float4 o[U][N];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int w = w0 + u * kSplit;
                v[u] = make_float2(-INFINITY, 0.f);
                if (w <= jn.last) v[u] = p.ml[slot(w)];
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int d = 4 * (lane + 32 * n);
                    o[u][n] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (w <= jn.last && d < D)
                        o[u][n] = *reinterpret_cast<const float4 *>(p.part + slot(w) * D + d);
                }
            }
            float top = m;
#pragma unroll
            for (int u = 0; u < U; ++u) top = fmaxf(top, v[u].x);
            const float old = m == top || m == -INFINITY ? (m == top ? 1.f : 0.f) : exp2_fast(m - top);
            m = top;
            l *= old;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                acc[n].x *= old;
                acc[n].y *= old;
                acc[n].z *= old;
                acc[n].w *= old;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float f = v[u].x == -INFINITY ? 0.f : v[u].x == m ? 1.f : exp2_fast(v[u].x - m);
                l += f * v[u].y;
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    acc[n].x += f * o[u][n].x;
                    acc[n].y += f * o[u][n].y;
                    acc[n].z += f * o[u][n].z;
                    acc[n].w += f * o[u][n].w;
                }
            }
        }
    }
    if constexpr (kSplit > 1) {
        if (lane == 0) sh_ml[warp] = make_float2(m, l);
#pragma unroll
        for (int n = 0; n < N; ++n) sh_o[warp][lane + 32 * n] = acc[n];
        __syncthreads();
        if (sub != 0) return;
        float top = m;
#pragma unroll
        for (int w = 0; w < kSplit; ++w) top = fmaxf(top, sh_ml[warp + w].x);
        l = 0.f;
#pragma unroll
        for (int n = 0; n < N; ++n) acc[n] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kSplit; ++w) {
            const float2 v = sh_ml[warp + w];
            const float f = v.x == -INFINITY ? 0.f : v.x == top ? 1.f : exp2_fast(v.x - top);
            l += f * v.y;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const float4 o = sh_o[warp + w][lane + 32 * n];
                acc[n].x += f * o.x;
                acc[n].y += f * o.y;
                acc[n].z += f * o.z;
                acc[n].w += f * o.w;
            }
        }
    }
    if (!live) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int h = jn.head * p.G + (R - i * p.G);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int d = 4 * (lane + 32 * n);
        if (d < D)
            store_out4(p, jn.row0 + i, h, d,
                       make_float4(acc[n].x * inv, acc[n].y * inv, acc[n].z * inv,
                                   acc[n].w * inv));
    }
}

}  // namespace tree
}  // namespace rarn
