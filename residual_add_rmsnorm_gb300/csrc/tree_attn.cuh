// tree_attn.cuh -- attention of drafted tokens over the paged 8-bit cache.
//
//   s_ij = scale * (q_i . K_j) * ks_j          over the visible j
//   o_i  = sum_j 2^(s_ij - m_i) vs_j V_j / sum_j 2^(s_ij - m_i)
//
// A sequence's keys are its context, which every drafted token sees, and its
// drafted tokens, of which token i sees those whose bit is set in its mask
// row (without a mask: those up to itself).  The G = Hq / Hk query heads that
// share a key head and a sequence's drafted tokens form the rows of one
// product, so each cached byte is read once for all of them.
//
// Work split.  A segment is one sequence, one key head and one block of rows;
// its keys form tiles of kTile.  All segments' tiles lie on one line, and CTA
// w of W takes the w-th equal part of it, whatever the sequences' lengths: a
// part that covers a segment wholly writes its rows' result, and the others
// leave (m, l, O) in the workspace for k_tree_join, which adds them in tile
// order (no atomics: the same inputs give the same bits).  Lengths are read
// on the device, so a captured call follows them.
#pragma once

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
    float scale_log2;        // scale * log2(e)
    // workspace
    int4 *joins;             // [segments]: first CTA, last CTA (-1: nothing to add), sequence,
                             // segment of that sequence
    int *count;              // segments of this call
    int max_segs;            // room in joins
    float2 *ml;              // [2 W][rows]
    float *part;             // [2 W][rows][D]
    unsigned int *watchdog;
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

__device__ __forceinline__ int64_t units_of(const Params &p, const Seq &s) {
    return (int64_t)p.cache.heads * s.blocks * s.tiles;
}

// Where a CTA's part of the line begins.
struct Cursor {
    int64_t total;   // tiles on the line
    int64_t lo, hi;  // this CTA's part
    int parts;       // CTAs with a part
    int b;           // sequence of lo
    int64_t base;    // first tile of that sequence on the line
    int seg0;        // segments before that sequence
};

// Prefix sums over the sequences by the whole CTA: thread i takes the i-th
// run of consecutive ones.  `sh` holds kN + 8 words of 8 bytes.
template <int kN>
__device__ __forceinline__ Cursor find_part(const Params &p, int rows, int tile, int64_t *sh) {
    const int run = (p.B + kN - 1) / kN;
    const int b0 = threadIdx.x * run, b1 = min(b0 + run, p.B);
    int64_t mine = 0, segs = 0;
    if (threadIdx.x < kN)
        for (int b = b0; b < b1; ++b) {
            const Seq s = seq_of(p, b, rows, tile);
            mine += units_of(p, s);
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
    const bool sound = gtotal <= p.max_segs;
    if (!sound) total = 0;
    Cursor c;
    c.total = total;
    c.parts = total < gridDim.x ? (int)total : (int)gridDim.x;
    const int w = blockIdx.x;
    c.lo = w < c.parts ? total * w / c.parts : total;
    c.hi = w < c.parts ? total * (w + 1) / c.parts : total;
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
            const int64_t n = units_of(p, s);
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
    c.base = sh[2 * kW + 1];
    c.seg0 = (int)sh[2 * kW + 2];
    return c;
}

// The last CTA whose part reaches into the tiles before `end`.
__device__ __forceinline__ int last_part(int64_t end, int64_t total, int parts) {
    // smallest z with total * (z + 1) / parts >= end
    int64_t z = (end * parts + total - 1) / total - 1;
    while (z > 0 && total * z / parts >= end) --z;
    while (total * (z + 1) / parts < end) ++z;
    return (int)z;
}

// A key's place in the cache: code and scale offsets of (its page, its slot),
// head included; code < 0: no such page.
struct KeyAt {
    int64_t code, scale;
};

__device__ __forceinline__ KeyAt key_at(const Params &p, int b, int head, int j, int len) {
    KeyAt k{-1, 0};
    if (j >= len) return k;
    const int pg = j / p.cache.page_size;
    const int at = j - pg * p.cache.page_size;
    const int64_t page = p.table[b * p.table_stride + pg];
    if (page < 0 || page >= p.cache.pages) {
        atomicOr(p.watchdog, kv::kWatchIndex);
        return k;
    }
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

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
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

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    return __byte_perm(a, b, sel);
}

// N 32-bit words from an address aligned to 4 N bytes, or to 16 where N is a
// multiple of 4.
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t *src) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = ld_stream(src + 4 * i);
            w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
        }
    } else if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(src + 4 * i);
            w[i] = v.x; w[i + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const uint32_t *>(src + 4 * i);
    }
}

// What a warp holds of kStep keys: the codes of keys g and g + 8 (its quarter
// of the row, for S = K Q^T) and of keys 2c, 2c + 1, 2c + 8, 2c + 9 (its
// eighth of the row, for O = V^T P), and the scales of keys g and g + 8.
template <int D>
struct Step {
    uint32_t k[2][D / 16];
    uint32_t v[4][D / 32];
    float ks[2], vs[2];
    uint32_t ok;  // bit j: key j of the step exists
};

template <int D>
__device__ __forceinline__ void load_step(const Params &p, Step<D> &st, int b, int head, int j0,
                                          int len) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    // lanes 0 .. 15 find their key's place; the others take it by shuffle
    const KeyAt mine = key_at(p, b, head, j0 + (lane & 15), len);
    st.ok = __ballot_sync(0xffffffffu, mine.code >= 0) & 0xffffu;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = g + 8 * h;
        const int64_t at = __shfl_sync(0xffffffffu, mine.code, j);
        const int64_t sc = __shfl_sync(0xffffffffu, mine.scale, j);
        if (at >= 0) {
            load_words(st.k[h], p.cache.k + at + c * (D / 4));
            st.ks[h] = p.cache.k_scale[sc];
            st.vs[h] = p.cache.v_scale[sc];
        } else {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) st.k[h][i] = 0;
            st.ks[h] = st.vs[h] = 0.f;
        }
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const int j = 2 * c + (h & 1) + (h >> 1) * 8;
        const int64_t at = __shfl_sync(0xffffffffu, mine.code, j);
        if (at >= 0) {
            load_words(st.v[h], p.cache.v + at + g * (D / 8));
        } else {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) st.v[h][i] = 0;
        }
    }
}

// Slack of the running maximum, in powers of two: a row's weights may reach
// 2^kSlack before its sums are rescaled, so that a rescale (a reduction over
// the warp and a pass over the accumulators) is rare.
constexpr float kSlack = 3.f;
// Weights enter the second product in binary16 as p vs / ref * 2^12, at most
// 2^15: what falls under 2^-24 of that, 2^-36 of the largest term, is lost,
// which 2^20 keys cannot add up to a rounding of the result.
constexpr float kWeightScale = 4096.f;

// A warp's running softmax and accumulators.
template <int D, int NQ, bool kE5M2>
struct RowState {
    float m[NQ][2];    // running maximum of the lane's rows (log2 units), -inf: none yet
    float l[NQ][2];    // this lane's keys' sum of weights
    float ref;         // the largest |vs| met, by which weights are divided
    float o[D / 16][NQ][4];

    __device__ __forceinline__ void clear() {
        ref = 1e-30f;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
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

// One segment's geometry, and what a lane needs to mask its four weights per
// row tile: the token and mask row of its rows.
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

// Values that are NaN or infinite and not visible to every row: in the second
// product 0 times such a value would be NaN, so those keys leave it (their
// codes become zero) and are added here to the rows that see them.  x: this
// lane's weights of keys g, g + 8; hidden: its bits.
template <int D, int NQ, bool kE5M2>
__device__ __forceinline__ void add_nonfinite(Step<D> &st, uint32_t keys, const float (&x)[NQ][4],
                                           uint32_t hidden, RowState<D, NQ, kE5M2> &rs) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll 1
    for (int j = 0; j < kStep; ++j) {
        if (!((keys >> j) & 1u)) continue;
        const int from = 4 * (j & 7) + c;
        const uint32_t hid = __shfl_sync(0xffffffffu, hidden, from);
        float w[NQ][2];
        bool vis[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                w[n][e] = __shfl_sync(0xffffffffu, j < 8 ? x[n][e] : x[n][2 + e], from);
                vis[n][e] = !((hid >> (4 * n + (j < 8 ? e : 2 + e))) & 1u);
            }
        const int which = (j & 1) + 2 * (j >> 3);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint32_t mine = which == 0 ? st.v[0][i] : which == 1 ? st.v[1][i]
                                                    : which == 2 ? st.v[2][i] : st.v[3][i];
            const uint32_t word = __shfl_sync(0xffffffffu, mine, 4 * g + ((j & 7) >> 1));
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float2 f = DT<__half>::w2f(
                    kv::codes2_to_h2<kE5M2>(u ? word >> 16 : word & 0xffffu));
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (vis[n][e]) {
                            rs.o[2 * i + u][n][e] += w[n][e] * f.x;
                            rs.o[2 * i + u][n][2 + e] += w[n][e] * f.y;
                        }
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 4; ++h)
        if ((keys >> (2 * c + (h & 1) + (h >> 1) * 8)) & 1u) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) st.v[h][i] = 0;
        }
}

template <int D, int NQ, bool kE5M2>
__device__ __forceinline__ void consume_step(const Params &p, const Segment &sg, Step<D> &st, int j0,
                                             const uint32_t (&q)[D / 16][NQ][2],
                                             const float (&cs)[NQ][2],
                                             RowState<D, NQ, kE5M2> &rs) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    float s[NQ][4];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        const uint32_t a0 = kv::codes2_to_h2<kE5M2>(st.k[0][i] & 0xffffu);
        const uint32_t a2 = kv::codes2_to_h2<kE5M2>(st.k[0][i] >> 16);
        const uint32_t a1 = kv::codes2_to_h2<kE5M2>(st.k[1][i] & 0xffffu);
        const uint32_t a3 = kv::codes2_to_h2<kE5M2>(st.k[1][i] >> 16);
#pragma unroll
        for (int n = 0; n < NQ; ++n) mma_16816(s[n], a0, a1, a2, a3, q[i][n][0], q[i][n][1]);
    }
    // s[n][0..1]: key g, rows 2c, 2c + 1; s[n][2..3]: key g + 8
    float top[NQ][2];
    const bool edge = st.ok != 0xffffu || j0 + kStep > sg.s.ctx;  // uniform
    uint32_t hidden = 0;  // bit 4 n + i: s[n][i] is not visible
    if (edge) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = g + 8 * h, d = j0 + j - sg.s.ctx;
            const bool exists = (st.ok >> j) & 1u;
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    int i, hq;
                    const bool live = row_of(p, sg, 8 * NQ, 8 * n + 2 * c + e, i, hq);
                    const bool vis =
                        exists && live && (d < 0 || sees(p, sg.row0 + i, i, d));
                    if (!vis) hidden |= 1u << (4 * n + 2 * h + e);
                }
        }
    }
    bool grow = false;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[n][i] = s[n][i] * (st.ks[i >> 1] * cs[n][i & 1]);
            if (edge && ((hidden >> (4 * n + i)) & 1u)) s[n][i] = -INFINITY;
        }
        top[n][0] = fmaxf(s[n][0], s[n][2]);
        top[n][1] = fmaxf(s[n][1], s[n][3]);
        grow |= top[n][0] > rs.m[n][0] + kSlack || top[n][1] > rs.m[n][1] + kSlack;
    }
    const float v0 = fabsf(st.vs[0]), v1 = fabsf(st.vs[1]);
    const float vmax = fmaxf(v0 < INFINITY ? v0 : 0.f, v1 < INFINITY ? v1 : 0.f);
    grow |= vmax > rs.ref;
    if (__any_sync(0xffffffffu, grow)) {
        float vm = max_over_keys(vmax);  // the same in every c
        const float ref = vm > rs.ref ? 2.f * vm < INFINITY ? 2.f * vm : vm : rs.ref;
        const float rr = rs.ref / ref;
        rs.ref = ref;
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float m = fmaxf(rs.m[n][e], max_over_keys(top[n][e]));
                const float a = rs.m[n][e] == m ? 1.f : exp2f(rs.m[n][e] - m);
                rs.m[n][e] = m;
                rs.l[n][e] *= a;
#pragma unroll
                for (int t = 0; t < D / 16; ++t) {
                    rs.o[t][n][e] *= a * rr;
                    rs.o[t][n][2 + e] *= a * rr;
                }
            }
    }
    const float inv_ref = kWeightScale / rs.ref;
    const float w0 = st.vs[0] * inv_ref, w1 = st.vs[1] * inv_ref;
    uint32_t pb[NQ][2];
    float x[NQ][4];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float m = rs.m[n][i & 1];
            const float pr = exp2f(s[n][i] - (m == -INFINITY ? 0.f : m));
            rs.l[n][i & 1] += pr;
            x[n][i] = pr * (i < 2 ? w0 : w1);
            if (edge && ((hidden >> (4 * n + i)) & 1u)) x[n][i] = 0.f;
        }
        pb[n][0] = transpose_8x8(pack_h2(x[n][0], x[n][1]));
        pb[n][1] = transpose_8x8(pack_h2(x[n][2], x[n][3]));
    }
    if (edge) {
        uint32_t bad = 0;  // this lane's keys with a value that is not finite
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            bool any = false;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) any |= any_nonfinite<kE5M2>(st.v[h][i]);
            if (any) bad |= 1u << (2 * c + (h & 1) + (h >> 1) * 8);
        }
        bad = __reduce_or_sync(0xffffffffu, bad);
        if (bad) add_nonfinite<D, NQ, kE5M2>(st, bad, x, hidden, rs);
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        // bytes of two keys interleaved: two elements per 32-bit word
        const uint32_t lo0 = prmt(st.v[0][i], st.v[1][i], 0x5140);
        const uint32_t lo1 = prmt(st.v[0][i], st.v[1][i], 0x7362);
        const uint32_t hi0 = prmt(st.v[2][i], st.v[3][i], 0x5140);
        const uint32_t hi1 = prmt(st.v[2][i], st.v[3][i], 0x7362);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t lo = u ? lo1 : lo0, hi = u ? hi1 : hi0;
            const uint32_t a0 = kv::codes2_to_h2<kE5M2>(lo & 0xffffu);
            const uint32_t a1 = kv::codes2_to_h2<kE5M2>(lo >> 16);
            const uint32_t a2 = kv::codes2_to_h2<kE5M2>(hi & 0xffffu);
            const uint32_t a3 = kv::codes2_to_h2<kE5M2>(hi >> 16);
#pragma unroll
            for (int n = 0; n < NQ; ++n)
                mma_16816(rs.o[2 * i + u][n], a0, a1, a2, a3, pb[n][0], pb[n][1]);
        }
    }
}

// The block's query rows as the second operand of S = K Q^T, in binary16, each
// row divided by a power of two that brings its largest magnitude to
// [2^13, 2^14): exact for bfloat16 except where an element is under 2^-27 of
// its row's largest.  cs: what undoes that, times the softmax scale, for the
// lane's rows 2c, 2c + 1.
template <int D, int NQ>
__device__ __forceinline__ void load_queries(const Params &p, const Segment &sg,
                                             uint32_t (&q)[D / 16][NQ][2], float (&cs)[NQ][2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        int i, h;
        const bool live = row_of(p, sg, 8 * NQ, 8 * n + g, i, h);
        float f[D / 4];
        float amax = 0.f;
        const int64_t at = (sg.row0 + i) * p.q.ts + (int64_t)h * p.q.hs + c * (D / 4);
#pragma unroll
        for (int e = 0; e < D / 4; e += 8) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (live) w = ld_stream(static_cast<const uint16_t *>(p.q.data) + at + e);
            float x[8];
            if (p.bf16) DT<__nv_bfloat16>::unpack(w, x);
            else DT<__half>::unpack(w, x);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                f[e + u] = x[u];
                amax = fmaxf(amax, fabsf(x[u]));
            }
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        int ex = amax > 0.f && amax < INFINITY ? ilogbf(amax) : 13;
        ex = ex < -100 ? -100 : ex;
        const float by = ldexpf(1.f, 13 - ex), back = ldexpf(1.f, ex - 13) * p.scale_log2;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            q[s][n][0] = pack_h2(f[4 * s] * by, f[4 * s + 1] * by);
            q[s][n][1] = pack_h2(f[4 * s + 2] * by, f[4 * s + 3] * by);
        }
        cs[n][0] = __shfl_sync(0xffffffffu, back, 8 * c);
        cs[n][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
    }
}

__device__ __forceinline__ void store_out(const Params &p, int64_t token, int h, int d, float v) {
    const int64_t at = token * p.out.ts + (int64_t)h * p.out.hs + d;
    if (p.bf16) static_cast<__nv_bfloat16 *>(p.out.data)[at] = __float2bfloat16_rn(v);
    else static_cast<__half *>(p.out.data)[at] = __float2half_rn(v);
}

// Four warps share a segment's tiles, kStep keys each in turn, with their own
// running maxima and sums; they are joined through shared memory at the end of
// the CTA's share of the segment.
template <int D, int NQ, bool kE5M2, bool kAhead>
__global__ void __launch_bounds__(kThreads) k_tree_rows(const Params p) {
    constexpr int kRows = 8 * NQ;
    constexpr int kPad = D + 4;  // floats per row of the join buffer
    __shared__ int64_t sh_part[kThreads + 8];
    __shared__ float sh_m[kWarps][kRows], sh_l[kWarps][kRows];
    __shared__ __align__(16) float sh_o[kWarps][kRows][kPad];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    grid_dependency_wait();
    grid_launch_dependents();
    const Cursor cur = find_part<kThreads>(p, kRows, kTile, sh_part);
    int64_t at = cur.lo, base = cur.base;
    int seg0 = cur.seg0;
    Segment sg;
    sg.b = cur.b;
    while (at < cur.hi) {
        sg.s = seq_of(p, sg.b, kRows, kTile);
        const int64_t units = units_of(p, sg.s);
        if (at >= base + units) {
            base += units;
            seg0 += p.cache.heads * sg.s.blocks;
            ++sg.b;
            continue;
        }
        const int64_t rel = at - base;
        const int which = (int)(rel / sg.s.tiles);
        const int t0 = (int)(rel - (int64_t)which * sg.s.tiles);
        const int64_t left = cur.hi - at;
        const int t1 = left < sg.s.tiles - t0 ? t0 + (int)left : sg.s.tiles;
        sg.head = which / sg.s.blocks;
        sg.block = which - sg.head * sg.s.blocks;
        sg.row0 = p.starts[sg.b];

        uint32_t q[D / 16][NQ][2];
        float cs[NQ][2];
        load_queries<D, NQ>(p, sg, q, cs);
        RowState<D, NQ, kE5M2> rs;
        rs.clear();
        const int j1 = min(t1 * kTile, sg.s.len);
        int j = t0 * kTile + warp * kStep;
        if constexpr (kAhead) {
            Step<D> now, next;
            if (j < j1) load_step<D>(p, now, sg.b, sg.head, j, sg.s.len);
            for (; j < j1; j += kTile) {
                const bool more = j + kTile < j1;
                if (more) load_step<D>(p, next, sg.b, sg.head, j + kTile, sg.s.len);
                consume_step<D, NQ, kE5M2>(p, sg, now, j, q, cs, rs);
                if (more) now = next;
            }
        } else {
            Step<D> now;
            for (; j < j1; j += kTile) {
                load_step<D>(p, now, sg.b, sg.head, j, sg.s.len);
                consume_step<D, NQ, kE5M2>(p, sg, now, j, q, cs, rs);
            }
        }
        // join the warps
        __syncthreads();  // the last segment's readers are done
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float l = sum_over_keys(rs.l[n][e]);
                if (g == 0) {
                    sh_m[warp][8 * n + 2 * c + e] = rs.m[n][e];
                    sh_l[warp][8 * n + 2 * c + e] = l;
                }
            }
        const float unit = rs.ref / kWeightScale;
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int t = 0; t < D / 16; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sh_o[warp][8 * n + 2 * c + (i & 1)][g * (D / 8) + 2 * t + (i >> 1)] =
                        rs.o[t][n][i] * unit;
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
                const float4 o = *reinterpret_cast<const float4 *>(&sh_o[w][r][d]);
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
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        store_out(p, sg.row0 + i, h, d + u, acc[u] * inv);
                }
            } else {
                if (d == 0) p.ml[slot * kRows + r] = make_float2(m, l);
                *reinterpret_cast<float4 *>(p.part + (slot * kRows + r) * D + d) =
                    make_float4(acc[0], acc[1], acc[2], acc[3]);
            }
        }
        if (t0 == 0 && threadIdx.x == 0)
            p.joins[seg0 + which] = make_int4(
                blockIdx.x, whole ? -1 : last_part(at + sg.s.tiles, cur.total, cur.parts), sg.b,
                which);
        at += t1 - t0;
    }
}

// Adds the parts of the segments that no CTA covered wholly, in tile order: a
// CTA per segment and 8 rows.
template <int D>
__global__ void __launch_bounds__(256) k_tree_join(const Params p, int rows, int tile) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int seg = blockIdx.x;
    if (seg >= *p.count) return;
    const int4 jn = p.joins[seg];
    if (jn.y < 0) return;
    Segment sg;
    sg.b = jn.z;
    sg.s = seq_of(p, sg.b, rows, tile);
    sg.head = jn.w / sg.s.blocks;
    sg.block = jn.w - sg.head * sg.s.blocks;
    sg.row0 = p.starts[sg.b];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.y * 8 + warp;
    int i, h;
    if (r >= rows || !row_of(p, sg, rows, r, i, h)) return;
    // the first part is in its CTA's slot 1, the later ones in slot 0
    auto slot = [&](int w) { return (2 * (int64_t)w + (w == jn.x ? 1 : 0)) * rows + r; };
    float m = -INFINITY;
    for (int w = jn.x + lane; w <= jn.y; w += 32) m = fmaxf(m, p.ml[slot(w)].x);
    m = warp_max(m);
    float l = 0.f;
    constexpr int N = (D + 127) / 128;
    float4 acc[N];
#pragma unroll
    for (int n = 0; n < N; ++n) acc[n] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int w = jn.x; w <= jn.y; ++w) {
        const int64_t s = slot(w);
        const float2 v = p.ml[s];
        const float f = v.x == -INFINITY ? 0.f : v.x == m ? 1.f : exp2f(v.x - m);
        l += f * v.y;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int d = 4 * (lane + 32 * n);
            if (d < D) {
                const float4 o = *reinterpret_cast<const float4 *>(p.part + s * D + d);
                acc[n].x += f * o.x;
                acc[n].y += f * o.y;
                acc[n].z += f * o.z;
                acc[n].w += f * o.w;
            }
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int d = 4 * (lane + 32 * n);
        if (d < D) {
            store_out(p, sg.row0 + i, h, d, acc[n].x * inv);
            store_out(p, sg.row0 + i, h, d + 1, acc[n].y * inv);
            store_out(p, sg.row0 + i, h, d + 2, acc[n].z * inv);
            store_out(p, sg.row0 + i, h, d + 3, acc[n].w * inv);
        }
    }
}

}  // namespace tree
}  // namespace rarn
