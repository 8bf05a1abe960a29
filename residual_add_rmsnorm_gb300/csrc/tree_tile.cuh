// tree_tile.cuh -- the attention of tree_attn.cuh for many rows per key head:
// 128 or 256 rows (drafted tokens x query heads of a group) against tiles of
// 128 keys on the fifth-generation tensor cores.
//
//   S = Q K^T    the keys' codes as they are, against the queries split into
//                e4m3 pieces (two hold a bfloat16, three a binary16), 8-bit
//                operands, binary32 sums
//   O = P V      binary16 operands, binary32 sums; P = 2^(s - m) vs
//
// With more than a few dozen rows mma.sync's rate (a quarter of tcgen05's) and
// the second product's conversions, which every block of rows makes anew,
// become the bound of k_tree_rows; here the values become binary16 once per
// tile in shared memory, whatever the number of rows, and the keys never.
//
// One CTA per SM, persistent over its part of the line of tiles:
//   * one warp looks up pages and copies codes by TMA, the keys' straight into
//     their operand's swizzled rows, a few tiles ahead; it puts the tile's
//     scales beside them.  Boxes are as large as the pages allow: the warp's
//     time per box bounds it with boxes of eight slots (one context of 131072
//     keys in pages of 64: 137 us, with boxes of 64 slots 123);
//   * four warps convert the values' codes (exactly) into an operand;
//   * two pipelines of four softmax warps take a tile in two passes of 64
//     keys: scores from tensor memory, weights rounded to binary16 over the
//     scores' columns;
//   * a warp for each pipeline issues its tcgen05.mma: S into one of the
//     pipeline's two times 64 columns, and O += P V with P read from tensor
//     memory.  S is a pass ahead of the softmax, which so never waits for the
//     products of its own pass, and issuing them, which takes as long as a
//     pass, keeps nobody (with both done in line by one of the softmax warps
//     16 sequences of drafted trees took 159 us, with the passes alone 179,
//     with the warp as well 126).
// With up to 128 rows the pipelines take alternate tiles of the same rows, and
// their states are joined at the end; with up to 256 rows each has its own
// 128.
//
// Code that runs once per tile is kept in rolled loops: the roles share an SM's
// instruction cache (16 sequences of drafted trees with the converters' loop unrolled by
// 8, 4, 1: 138, 126, 124 us; one context of 131072 keys: 129, 122, 116).
//
// Every wait is bounded; one that runs out sets watchdog bit 5, the CTA's
// warps give up together, its segments' records say so (give_up), and its
// tensor memory is freed.
#pragma once

#include <cstddef>

#include "tree_attn.cuh"
#include "tree_offset.h"
#include "tree_plan.h"

namespace rarn {
namespace tree {

constexpr int kTileKeys = 128;   // keys of a tile
static_assert(kTileKeys != kTile, "begin_units tells the kernels apart");
constexpr int kTileRows = 128;   // rows of a pipeline
constexpr int kPass = 64;        // keys of a pass of the softmax, half a tile
constexpr int kBox = kBoxSlots;  // slots of the smallest TMA box
constexpr int kSoftWarps = 8;
constexpr int kConvWarps = 4;
constexpr int kIssueWarps = 2;   // of a pipeline's products
constexpr int kTileThreads = 32 * (kSoftWarps + kConvWarps + 1 + kIssueWarps);
constexpr int kMaxTileCtas = 160;
constexpr int kInfos = 8;        // tiles whose scales are kept
constexpr float kLiftSlack = 2.f;

// What the softmax needs of a tile besides its scores.
struct TileInfo {
    float kk[kTileKeys];  // key scale x softmax scale (log2 units), 0 where there is no key
    float vs[kTileKeys];  // value scale, 0 where there is no key
    uint32_t ok[4];       // keys that exist
    // of each pass's keys: lift_of the largest finite |vs|, and whether others'
    // are more than kLiftSlack under it
    float lift[2];
    float wide[2];  // 1 or 0
};

// Shared memory: the queries' pieces (over which pipeline 1's state is laid
// for the join), rings of the keys' and the values' codes, two converted
// value tiles, the tiles' scales.
template <int D, int NP, bool kTwo>
struct TileSmem {
    static constexpr int kCodes = kTileKeys * D;       // bytes of a tile's codes
    static constexpr int kHalf = 2 * kCodes;           // in binary16
    static constexpr int kQ = 0;
    static constexpr int kQBytes = kTwo ? 2 * NP * kCodes : 4 * kCodes;
    static constexpr int kStagesK = kTwo && NP == 3 ? 2 : 3;
    static constexpr int kStagesV = kTwo && NP == 3 ? 1 : 2;
    static constexpr int kK = kQ + kQBytes;
    static constexpr int kV = kK + kStagesK * kCodes;
    static constexpr int kVh = kV + kStagesV * kCodes;
    static constexpr int kInfo = kVh + 2 * kHalf;
    static constexpr int kBytes = kInfo + kInfos * (int)sizeof(TileInfo) + 1024;
    static_assert(4 * kCodes >= kTileRows * D * 4 || kTwo, "room for the join");
};

// Barriers, in one array.
enum Bar : int {
    B_KFULL = 0, B_KEMPTY = 3, B_VFULL = 6, B_VEMPTY = 8, B_HFULL = 10, B_HEMPTY = 12,
    B_SFULL = 14, B_PFULL = 18, B_ODONE = 22, B_QREADY = 26, B_INFO = 28, B_MERGE = 36,
    B_QDONE = 37, B_NEXT = 38, B_DRAIN = 39, B_COUNT = 40
};

// A CTA's share of the line, segment by segment.  Every role walks it alike;
// the softmax warps, short of registers, keep theirs in shared memory.
struct Walk {
    int at, hi, base, seg0;
    Segment sg;
    int t0, t1, which;
    int last_unit;  // of the segment, on the line

    __device__ __forceinline__ void begin(const Cursor &c) {
        at = c.lo;
        hi = c.hi;
        base = c.base;
        seg0 = c.seg0;
        t0 = t1 = which = last_unit = 0;
        sg.b = c.b;
    }
    // The next segment; false when there is none.
    __device__ __forceinline__ bool next(const Params &p, int rows) {
        int a = at, bs = base, sb = sg.b, s0 = seg0;
        bool found = false;
        while (a < hi) {
            const Seq q = seq_of(p, sb, rows, kTileKeys);
            constexpr int kBegin = begin_units(kTileKeys);
            const int units = (int)units_of(p, q, kTileKeys);
            if (a < bs + units) {
                const int each = q.tiles + kBegin;
                const int w = (unsigned)(a - bs) / (unsigned)each;
                const int x0 = a - bs - w * each, x1 = min(x0 + hi - a, each);
                a += x1 - x0;
                const int first = max(x0 - kBegin, 0), end = x1 - kBegin;
                if (end <= first) continue;
                which = w;
                t0 = first;
                t1 = end;
                last_unit = a - x1 + each - 1;
                sg.s = q;
                const int head = (unsigned)w / (unsigned)q.blocks;
                sg.head = head;
                sg.block = w - head * q.blocks;
                sg.row0 = p.starts[sb];
                found = true;
                break;
            }
            bs += units;
            s0 += p.cache.heads * q.blocks;
            ++sb;
        }
        at = a;
        base = bs;
        seg0 = s0;
        sg.b = sb;
        return found;
    }
};

// Bounded wait; false when it or another warp's ran out.
__device__ __forceinline__ bool tile_wait(const Params &p, uint32_t bar, uint32_t parity,
                                          volatile int *abort_flag) {
    if (gemm::mbar_try_wait(bar, parity)) return true;
    unsigned long long t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (gemm::mbar_try_wait(bar, parity)) return true;
        if ((i & 127u) == 0) {
            if (*abort_flag) return false;
            const unsigned long long t = gemm::now_ns();
            if (t0 == 0) {
                t0 = t;
            } else if (t - t0 > p.wait_limit_ns) {
                *abort_flag = 1;
                atomicOr(p.watchdog, kWatchTree);
                return false;
            }
        }
    }
}

// Codes that are NaN or infinite become zero.
template <bool kE5M2>
__device__ __forceinline__ uint32_t finite_codes(uint32_t w) {
    constexpr uint32_t top = kE5M2 ? 0x7c7c7c7cu : 0x7f7f7f7fu;
    return w & ~__vcmpeq4(w & top, top);
}

// Byte of 16-byte chunk x of a row of codes, in the TMA swizzle of rows of D
// bytes; and of chunk c (8 elements) of a row of `half` 64 binary16 elements.
template <int D>
__device__ __forceinline__ uint32_t code_at(int row, int x) {
    return row * D + ((x ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4);
}

__device__ __forceinline__ uint32_t half_at(int row, int half, int c) {
    return half * (kTileKeys * 128) + row * 128 + ((c ^ (row & 7)) << 4);
}

// V as the N-major operand: 64-element blocks of N lie kTileKeys rows apart,
// groups of eight keys 1024 bytes.
__device__ __forceinline__ uint64_t value_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((kTileKeys * 128) >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// Instruction descriptors: 8-bit operands of e4m3 (0) by e4m3 or e5m2 (1), and
// binary16 with an N-major second operand.
template <bool kE5M2>
__host__ __device__ constexpr uint32_t scores_desc() {
    return (1u << 4) | (0u << 7) | ((kE5M2 ? 1u : 0u) << 10) |
           ((uint32_t)(kPass >> 3) << 17) | ((uint32_t)(kTileRows >> 4) << 24);
}

template <int N>
__host__ __device__ constexpr uint32_t products_desc() {
    return gemm::instr_desc<__half, N>() | (1u << 16);
}

__device__ __forceinline__ void mma_f8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The first operand in tensor memory.
__device__ __forceinline__ void mma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                           uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        "}\n" ::"r"(tmem_d),
        "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void st_global32f(float *p, const float (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]),
                 "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

// Columns [0, 32) of O scaled in place.
__device__ __forceinline__ void tmem_scale32(uint32_t taddr, float by) {
    float v[32];
    gemm::tmem_ld32(taddr, v);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t r[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[16 * h + i] * by);
        tmem_st16(taddr + 16 * h, r);
    }
}

// Which of the 32 keys from drafted token d0 (negative: context) on a row
// sees.
__device__ __forceinline__ uint32_t seen_word(const Params &p, int64_t row, int tok,
                                              int d0) {
    if (d0 + 31 < 0) return 0xffffffffu;
    if (!p.mask) {
        // tokens up to itself: bits 0 .. tok - d0
        const int last = tok - d0;
        return last >= 31 ? 0xffffffffu : last < 0 ? 0u : 0xffffffffu >> (31 - last);
    }
    auto word = [&](int w) {
        return w >= 0 && w < p.words ? p.mask[row * p.words + w] : 0u;
    };
    const int w = d0 >= 0 ? d0 >> 5 : -1, sh = d0 & 31;  // -1: the word of the context's end
    const uint32_t lo = d0 >= 0 ? word(w) : 0xffffffffu;
    return sh ? __funnelshift_r(lo, word(w + 1), sh) : lo;
}

// What the products left out: NaN and infinite values of drafted tokens
// behind key j0 and before j1, for one row that sees them, elements
// [e0, e0 + 32).
template <bool kE5M2>
__device__ __forceinline__ void add_nonfinite(const Params &p, const Segment &sg, int tok, int j0,
                                              int j1, int e0, float (&o)[32]) {
#pragma unroll 1
    for (int d = max(0, j0 - sg.s.ctx); d < sg.s.n; ++d) {
        const int j = sg.s.ctx + d;
        if (j >= j1 || j >= sg.s.len) break;
        if (!sees(p, sg.row0 + tok, tok, d)) continue;
        const int pg = p.page_of(j);
        const int64_t page = p.table[sg.b * p.table_stride + pg];
        if (page < 0 || page >= p.cache.pages) continue;
        const uint8_t *v =
            p.cache.v + place(p, page, j - pg * p.cache.page_size, sg.head).code + e0;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            const float2 x = DT<__half>::w2f(kv::codes2_to_h2<kE5M2>(v[e]));
            if (!(fabsf(x.x) < INFINITY)) o[e] += x.x;
        }
    }
}

// The softmax reads scores in fragments: of 16 rows and 8 columns a lane has
// columns 2c, 2c + 1 (c = lane % 4) of rows g and g + 8 (g = lane / 4).  A
// lane so meets a quarter of a tile's keys in each of four rows, not all of
// them in one, and the keys' factors, which every row needs, cost a quarter of
// the shared-memory reads that a row to a lane takes.
// 32 columns of 16 rows on their way to registers (4 i ..: columns 8 i ..).
__device__ __forceinline__ void tmem_frag_begin(uint32_t taddr, float (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
          "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]),
          "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr));
}

// The arrival of both halves of a warp's rows.
__device__ __forceinline__ void tmem_frag_end(float (&r)[16], float (&q)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]),
                   "+f"(r[6]), "+f"(r[7]), "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]),
                   "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])
                 :
                 : "memory");
    asm volatile(""
                 : "+f"(q[0]), "+f"(q[1]), "+f"(q[2]), "+f"(q[3]), "+f"(q[4]), "+f"(q[5]),
                   "+f"(q[6]), "+f"(q[7]), "+f"(q[8]), "+f"(q[9]), "+f"(q[10]), "+f"(q[11]),
                   "+f"(q[12]), "+f"(q[13]), "+f"(q[14]), "+f"(q[15])
                 :
                 : "memory");
}

// 16 columns of 16 rows: the same fragments as binary16 pairs.
__device__ __forceinline__ void tmem_frag_store(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ uint64_t lds64(uint32_t a) {
    uint64_t v;
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}

// Where a tile's figures are in shared memory.
constexpr uint32_t kInfoVs = offsetof(TileInfo, vs), kInfoOk = offsetof(TileInfo, ok),
                   kInfoLift = offsetof(TileInfo, lift), kInfoWide = offsetof(TileInfo, wide);

constexpr uint32_t kHalfRows = 16u << 16;  // tensor memory's address of a warp's second 16 rows

// Two binary32 values in one 64-bit register, and packed arithmetic on them.
__device__ __forceinline__ uint64_t two(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float2 apart(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// A value of each of a lane's four rows (g, g + 8, g + 16, g + 24) from or to
// the lane that owns the row (lane = row of the warp).
__device__ __forceinline__ void rows_from_owner(float own, float (&v)[4]) {
    const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xffffffffu, own, g + 8 * i);
}

__device__ __forceinline__ float rows_to_owner(const float (&v)[4]) {
    const int lane = threadIdx.x & 31;
    float own = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = __shfl_sync(0xffffffffu, v[i], 4 * (lane & 7));
        if ((lane >> 3) == i) own = x;
    }
    return own;
}

// The largest scores of a warp's 32 rows over a pass (S at `ts`, columns times
// the keys' factors at `ti`), each in the lane that owns the row.  kEdge: only
// where bits of v0, v1 (of the lane's own row) are set.  For rows without an
// offset.
template <bool kEdge>
__device__ __noinline__ float row_top(uint32_t ts, uint32_t ti, uint32_t v0, uint32_t v1,
                                      float back) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c2 = 2 * (lane & 3);
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
    for (int c = 0; c < kPass / 32; ++c) {
        float s[2][16];
        tmem_frag_begin(ts + 32 * c, s[0]);
        tmem_frag_begin(ts + 32 * c + kHalfRows, s[1]);
        uint64_t kk[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            kk[j] = lds64(ti + 4 * (32 * c + 8 * j + c2));
        const uint32_t word = kEdge ? (c ? v1 : v0) : 0u;
        tmem_frag_end(s[0], s[1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // row g + 8 i
            const uint32_t v = kEdge ? __shfl_sync(0xffffffffu, word, g + 8 * i) >> c2 : 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = 4 * j + 2 * (i & 1);
                float2 a = apart(mul2(two(s[i >> 1][at], s[i >> 1][at + 1]), kk[j]));
                if (kEdge) {
                    if (!((v >> (8 * j)) & 1u)) a.x = -INFINITY;
                    if (!((v >> (8 * j + 1)) & 1u)) a.y = -INFINITY;
                }
                top[i] = max3(top[i], a.x, a.y);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
    }
    return rows_to_owner(top) * back;
}

// A lane's row of the running softmax.  Weights are 2^(score - off), and with
// the value scale vs enter the products as binary16.  An offset is chosen when
// the row first sees a key, such that its largest weight times the tile's
// largest vs is 2^kCentre, and moves up only when one would pass 2^kHighest: a
// pass over the scores serves where finding their maximum first took two.
// What falls under 2^-24 of the product's units, 2^-25 of the row's largest
// weight times the largest value scale that it sees, is lost; 2^14 keys at that
// edge would add up to half of binary16's own rounding.
struct RowLane {
    float off;   // of the own row
    bool set;    // the offset is chosen (rows that are not there count as such)
    // of the four rows that the lane has fragments of: minus the offset, what
    // undoes the scaling of the row's query, and the sums over the lane's keys
    float sub[4], back[4];
    uint64_t l[4];
};

// ceil(log2) of a largest value scale, within what binary32 sums of weights
// bear.
__device__ __forceinline__ float lift_of(float vmax) {
    const int e = (int)(__float_as_uint(vmax) >> 23) - 126;
    return (float)max(-70, min(e, 100));
}

// Scales by 2^-down (a row to a lane) what the row has summed up: O (its D
// columns at `to`, where there is any), and the first `chunks` times 16 columns
// of binary16 weights at `ts`.
template <int D>
__device__ __noinline__ void scale_down(uint32_t to, bool any, uint32_t ts, int chunks,
                                        float down) {
    const float by = exp2_fast(-down);
    if (any) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) tmem_scale32(to + 32 * c, by);
    }
    // the pass's earlier weights are stored asynchronously, in another shape
    if (chunks) tmem_st_wait();
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        uint32_t w[16];
        tmem_ld16(ts + 16 * c, w);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 x = DT<__half>::w2f(w[i]);
            w[i] = pack_h2(x.x * by, x.y * by);
        }
        tmem_st16(ts + 16 * c, w);
    }
    tmem_st_wait();
}

// The same over the keys of a pass whose bits of v0, v1 are set (figures at
// `ti`).  Where a row does not see them all, a hidden token's scale must not
// choose its offset.
static __device__ __noinline__ float row_lift(uint32_t ti, uint32_t v0, uint32_t v1) {
    float most = 0.f;
#pragma unroll 1
    for (int c = 0; c < kPass / 2; ++c) {
        const uint32_t v = c < 16 ? v0 >> (2 * c) : v1 >> (2 * c - 32);
        const float2 s = apart(lds64(ti + kInfoVs + 8 * c));
        if ((v & 1u) && fabsf(s.x) < INFINITY) most = fmaxf(most, fabsf(s.x));
        if ((v & 2u) && fabsf(s.y) < INFINITY) most = fmaxf(most, fabsf(s.y));
    }
    return lift_of(most);
}

// moved_offset out of line, {sub, down}: rare, and the roles share an instruction
// cache.
static __device__ __noinline__ float2 move_offset(float sub, float high, float centre) {
    float2 r;
    r.x = moved_offset(sub, high, centre, &r.y);
    return r;
}

// The smaller; NaN where a is.
__device__ __forceinline__ float cut(float a, float most) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(most));
    return r;
}

// A warp's weights of a pass (S at `ts`, columns times the keys' factors at
// `ti`), in binary16 over the scores' columns.  `lift`: of the value scales
// that the own row sees.  Where a score is more than kHighest - lift over its
// row's offset, all that the row has so far is scaled down first, once the
// products under way are in (`settled`), so that it comes to kCentre - lift or
// up to one under it: by a power of two, which rounds no weight anew that stays
// normal in binary16.  This is done kMoves times at most for 32 keys, nearly
// always once; a score that is over even then is cut.
// kEdge: only keys whose bits of v0, v1 (the own row's) are set.
template <int D, bool kEdge, class Settled>
__device__ __forceinline__ bool row_weights(uint32_t ts, uint32_t to, bool any, uint32_t ti,
                                            uint32_t v0, uint32_t v1, float lift,
                                            RowLane &row, const Settled &settled) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c2 = 2 * (lane & 3);
    float most = kHighest - lift;  // the same for all rows within the context, else the least
    if (kEdge) {
        float m[4];
        rows_from_owner(most, m);
        most = fminf(fminf(m[0], m[1]), fminf(m[2], m[3]));
    }
    int moves = 0;  // of the offset, for these keys
#pragma unroll 1
    for (int c = 0; c < kPass / 32;) {
        float s[2][16];
        tmem_frag_begin(ts + 32 * c, s[0]);
        tmem_frag_begin(ts + 32 * c + kHalfRows, s[1]);
        uint64_t kk[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            kk[j] = lds64(ti + 4 * (32 * c + 8 * j + c2));
        const uint32_t word = kEdge ? (c ? v1 : v0) : 0u;
        tmem_frag_end(s[0], s[1]);
        float top[4];
        bool over = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // row g + 8 i
            const uint32_t v = kEdge ? __shfl_sync(0xffffffffu, word, g + 8 * i) >> c2 : 0u;
            const uint64_t shift = two(row.sub[i], row.sub[i]), by = two(row.back[i], row.back[i]);
            float high = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = 4 * j + 2 * (i & 1);
                float2 a = apart(
                    fma2(mul2(two(s[i >> 1][at], s[i >> 1][at + 1]), kk[j]), by, shift));
                if (kEdge) {
                    if (!((v >> (8 * j)) & 1u)) a.x = -INFINITY;
                    if (!((v >> (8 * j + 1)) & 1u)) a.y = -INFINITY;
                }
                s[i >> 1][at] = a.x;
                s[i >> 1][at + 1] = a.y;
                high = max3(high, a.x, a.y);
            }
            top[i] = high;
            over |= high > most;
        }
        if (__any_sync(0xffffffffu, over)) {
            // rare: the offset moves up under what is there; then again
            float limit[4];
            rows_from_owner(kHighest - lift, limit);
            over = top[0] > limit[0] || top[1] > limit[1] || top[2] > limit[2] ||
                   top[3] > limit[3];
            if (moves < kMoves && __any_sync(0xffffffffu, over)) {
                ++moves;
                float d[4], off[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float high = top[i];
                    high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, 1));
                    high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, 2));
                    d[i] = 0.f;
                    if (high > limit[i]) {
                        const float2 moved =
                            move_offset(row.sub[i], high, limit[i] - (kHighest - kCentre));
                        row.sub[i] = moved.x;
                        d[i] = moved.y;
                    }
                    off[i] = -row.sub[i];
                    const float q = exp2_fast(-d[i]);
                    row.l[i] = mul2(row.l[i], two(q, q));
                }
                const float down = rows_to_owner(d);
                row.off = rows_to_owner(off);
                if (any && !settled()) return false;
                scale_down<D>(to, any, ts, c, down);
                continue;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {  // of rows g, g + 8, and 16 more
                const int i = (j >> 1) & 1;
                s[0][j] = cut(s[0][j], limit[i]);
                s[1][j] = cut(s[1][j], limit[i + 2]);
            }
        }
        uint64_t vs[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            vs[j] = lds64(ti + kInfoVs + 4 * (32 * c + 8 * j + c2));
        uint32_t w[2][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = kEdge ? __shfl_sync(0xffffffffu, word, g + 8 * i) >> c2 : 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = 4 * j + 2 * (i & 1);
                const uint64_t pr =
                    two(exp2_fast(s[i >> 1][at]), exp2_fast(s[i >> 1][at + 1]));
                row.l[i] = add2(row.l[i], pr);
                float2 a = apart(mul2(pr, vs[j]));
                if (kEdge) {
                    if (!((v >> (8 * j)) & 1u)) a.x = 0.f;
                    if (!((v >> (8 * j + 1)) & 1u)) a.y = 0.f;
                }
                w[i >> 1][2 * j + (i & 1)] = pack_h2(a.x, a.y);
            }
        }
        tmem_frag_store(ts + 16 * c, w[0]);  // over columns that are read
        tmem_frag_store(ts + 16 * c + kHalfRows, w[1]);
        moves = 0;
        ++c;
    }
    return true;
}

// A CTA whose waits ran out: k_tree_join finds no segment that began here, whose
// record may not have been written, and NaN in what belongs to an earlier one.
inline __device__ __noinline__ void give_up(const Params &p, const Cursor &cur, int rows) {
    for (int x = threadIdx.x; x < 2 * rows; x += kTileThreads)
        p.ml[2 * (int64_t)blockIdx.x * rows + x] = make_float2(NAN, NAN);
    if (threadIdx.x != 0) return;
    Walk walk;
    walk.begin(cur);
    while (walk.next(p, rows))
        if (walk.t0 == 0)
            p.joins[walk.seg0 + walk.which] = Join{(int)blockIdx.x, -1, 0, 0, 0, 0, 0, 0};
}

// The sum of weights of the lane's own row.
__device__ __forceinline__ float row_sum(const RowLane &row) {
    float sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = apart(row.l[i]);
        sum[i] = x.x + x.y;
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
    }
    return rows_to_owner(sum);
}

// kTwo: 256 rows, 128 to each pipeline; else 128, tiles alternate.  NP: pieces
// of a query.
template <int D, int NP, bool kE5M2, bool kTwo>
__global__ void __launch_bounds__(kTileThreads, 1)
    k_tree_tile(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
    using S = TileSmem<D, NP, kTwo>;
    constexpr int kRows = kTwo ? 2 * kTileRows : kTileRows;
    constexpr uint32_t kTmemO = 256;  // O of pipeline 0; S are columns 0 and 128
    extern __shared__ uint8_t smem_raw[];
    __shared__ int64_t sh_part[16];
    __shared__ __align__(8) uint64_t sh_bar[B_COUNT];
    __shared__ uint32_t sh_tmem;
    __shared__ volatile int sh_abort;
    __shared__ volatile int sh_nonfinite;  // a value was kept out of the products
    __shared__ float sh_back[kRows];       // what undoes the scaling of a row's query
    __shared__ float2 sh_ml[kTileRows];    // pipeline 1's l and offset
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    TileInfo *info = reinterpret_cast<TileInfo *>(smem + S::kInfo);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t bars = smem_u32(sh_bar);
    auto bar = [&](int b) { return bars + 8 * b; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i) {
            // arrivals of one thread, of the four warps of a role, of the
            // products of each pipeline, or of all who begin a segment
            int n = 1;
            if ((i >= B_VEMPTY && i < B_HFULL + 2) || (i >= B_PFULL && i < B_ODONE) ||
                (i >= B_QREADY && i < B_INFO) || i == B_MERGE)
                n = 4;
            if (i == B_NEXT) n = kSoftWarps + 1;
            if ((i >= B_KEMPTY && i < B_VFULL) || (i >= B_HEMPTY && i < B_SFULL)) n = kTwo ? 2 : 1;
            if (i == B_DRAIN) n = 2;
            gemm::mbar_init(bar(i), n);
        }
        gemm::fence_async_shared();
        sh_abort = 0;
        sh_nonfinite = 0;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sh_tmem)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    gemm::tmem_fence_before();
    __syncthreads();
    gemm::tmem_fence_after();
    const uint32_t tmem = sh_tmem;
    grid_dependency_wait();
    grid_launch_dependents();
    const Cursor cur = find_part<128>(p, kRows, kTileKeys, sh_part);
    // for the softmax warps, short of registers: their first lanes', and thread 0's
    __shared__ Walk sh_walk[kSoftWarps];
    __shared__ Cursor sh_cur;
    if (threadIdx.x == 0) sh_cur = cur;

    if (warp == kSoftWarps + kConvWarps) {
        // ---------------- copies ----------------
        // The stream of tiles over all segments.  Lane b (and b + 16) knows
        // the page of slots 8 b .. 8 b + 7, lane l the scales of keys 4 l .. 4 l + 3.  Pages
        // are loaded two tiles ahead and scales one, or each tile would wait
        // for one load after the other.
        Walk walk;
        walk.begin(cur);
        int tile = 0;
        bool more = walk.next(p, kRows);
        if (more) tile = walk.t0;
        struct Next {
            int page, at, head, live;  // of the lane's slots; keys of the tile
            bool there;
        } nx, after;
        float ksc[4], vsc[4];  // of tile nx
        auto look = [&]() {   // nx becomes the tile behind, after the one behind that
            nx = after;
            after.there = more;
            if (more) {
                const Segment &sg = walk.sg;
                const int j0 = tile * kTileKeys, jb = j0 + kBox * (lane & 15);
                after.head = sg.head;
                after.live = sg.s.len - j0;
                after.page = -1;
                after.at = 0;
                if (jb < sg.s.len) {
                    after.page = p.table[sg.b * p.table_stride + p.page_of(jb)];
                    after.at = p.offset_in_page(jb);
                }
                if (++tile >= walk.t1) {
                    more = walk.next(p, kRows);
                    tile = walk.t0;
                }
            }
            if (!nx.there) return;
            if (kBox * (lane & 15) < nx.live && (nx.page < 0 || nx.page >= p.cache.pages)) {
                nx.page = -1;
                atomicOr(p.watchdog, kv::kWatchIndex);
            }
            const int page = __shfl_sync(0xffffffffu, nx.page, lane >> 1);
            const int at = __shfl_sync(0xffffffffu, nx.at, lane >> 1) + 4 * (lane & 1);
            const int64_t base = (int64_t)page * p.cache.s_page + nx.head * p.cache.s_head;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ksc[i] = vsc[i] = 0.f;
                if (page >= 0 && 4 * lane + i < nx.live) {
                    ksc[i] = p.cache.k_scale[base + (at + i) * p.cache.s_slot];
                    vsc[i] = p.cache.v_scale[base + (at + i) * p.cache.s_slot];
                }
            }
        };
        const int stall_at = blockIdx.x == 0 ? p.stall_fill : -1;
        // lanes whose eight slots are the first of a box
        const uint32_t first =
            __ballot_sync(0xffffffffu, lane < 16 && ((kBox * lane) & (p.box - 1)) == 0);
        auto copy = [&](const CUtensorMap *map, uint32_t dst, uint32_t full, uint32_t boxes,
                        const Next &x, int fill) {
            if (lane == 0)
                gemm::mbar_arrive_expect_tx(full, p.box * D * __popc(boxes & first) +
                                                      (fill == stall_at ? 16u : 0u));
            __syncwarp();
            if (((first >> lane) & 1u) && x.page >= 0)
                tma_box(dst + lane * (kBox * D), map, full, 0, x.at, x.head, x.page);
        };
        after.there = false;
        look();
        look();
        int nk = 0, nv = 0;    // fills
        int ks = 0, vs = 0;    // stages
        uint32_t kp = 1, vp = 1;     // parities of their releases
#pragma unroll 1
        for (int n = 0; nx.there; ++n) {
            const Next now = nx;
            const uint32_t boxes = __ballot_sync(0xffffffffu, now.page >= 0) & 0xffffu;
            bool alive = tile_wait(p, bar(B_KEMPTY + ks), kp, &sh_abort);
            if (!__all_sync(0xffffffffu, alive)) break;
            copy(&kmap, sbase + S::kK + ks * S::kCodes, bar(B_KFULL + ks), boxes, now,
                 2 * n);
            ++nk;
            if (++ks == S::kStagesK) {
                ks = 0;
                kp ^= 1;
            }
            // The scales.  The tile that had the place eight tiles ago is done
            // with: the products of tile n - 4 or later, which the release of
            // this stage of keys waited for, came after its softmax.
            TileInfo &ti = info[n & (kInfos - 1)];
            float vmax = 0.f, vmin = INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ti.kk[4 * lane + i] = ksc[i] * p.scale_log2;
                ti.vs[4 * lane + i] = vsc[i];
                const float a = fabsf(vsc[i]);
                if (a < INFINITY) vmax = fmaxf(vmax, a);
                if (a > 0.f) vmin = fminf(vmin, a);
            }
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) {  // over the half warp of a pass's keys
                vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, d));
                vmin = fminf(vmin, __shfl_xor_sync(0xffffffffu, vmin, d));
            }
            if (lane < 4) {
                uint32_t w = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if ((boxes >> (4 * lane + i)) & 1u) w |= 0xffu << (8 * i);
                const int left = now.live - 32 * lane;
                ti.ok[lane] = left >= 32 ? w : left <= 0 ? 0u : w & ((1u << left) - 1u);
            }
            if ((lane & 15) == 0) {
                const float lift = lift_of(vmax);
                ti.lift[lane >> 4] = lift;
                ti.wide[lane >> 4] = lift - lift_of(vmin) > kLiftSlack ? 1.f : 0.f;
            }
            __syncwarp();
            if (lane == 0) gemm::mbar_arrive(bar(B_INFO + (n & (kInfos - 1))));
            look();
            alive = tile_wait(p, bar(B_VEMPTY + vs), vp, &sh_abort);
            if (!__all_sync(0xffffffffu, alive)) break;
            copy(&vmap, sbase + S::kV + vs * S::kCodes, bar(B_VFULL + vs), boxes, now,
                 2 * n + 1);
            ++nv;
            if (++vs == S::kStagesV) {
                vs = 0;
                vp ^= 1;
            }
        }
        if (sh_abort && lane == 0) {
            // let what is under way land before the CTA goes, if it does
            const unsigned long long t0 = gemm::now_ns();
            auto landed = [&](int b, int fills, int stages) {
                for (int f = max(0, fills - stages); f < fills; ++f)
                    while (!gemm::mbar_try_wait(bar(b + f % stages), (f / stages) & 1) &&
                           gemm::now_ns() - t0 < p.wait_limit_ns) {
                    }
            };
            landed(B_KFULL, nk, S::kStagesK);
            landed(B_VFULL, nv, S::kStagesV);
        }
        __syncwarp();
    } else if (warp > kSoftWarps + kConvWarps) {
        // ---------------- a pipeline's products ----------------
        // In the order that keeps the tensor cores ahead of the softmax: the
        // scores of a pass are issued behind the products of the pass two
        // before, whose columns they take.
        const int pipe = warp - (kSoftWarps + kConvWarps + 1);
        Walk walk;
        walk.begin(cur);
        int n = 0;                    // tiles of finished segments
        int items = 0, segment = 0;   // items: tiles of this pipeline
        constexpr int kEach = kTwo ? 1 : 2;
        // Item t of a segment that began at tile n is key tile n + t.
        auto scores = [&](int t, int half, bool last) {
            const int stage = (n + t) % S::kStagesK;
            // The tile that had this stage before is the other pipeline's.  Were
            // it still on its way, the wait for this one's phase would take the
            // phase before that for it; the tile's figures come after the
            // release of the stage, and so after that tile.
            if (!kTwo && half == 0 &&
                !tile_wait(p, bar(B_INFO + ((n + t) & (kInfos - 1))), ((n + t) >> 3) & 1,
                           &sh_abort))
                return false;
            if (half == 0 &&
                !tile_wait(p, bar(B_KFULL + stage), ((n + t) / S::kStagesK) & 1, &sh_abort))
                return false;
            gemm::tmem_fence_after();
            const uint32_t qb = sbase + S::kQ + (kTwo ? pipe * NP * S::kCodes : 0);
            const uint32_t kb = sbase + S::kK + stage * S::kCodes + half * (kPass * D);
#pragma unroll
            for (int u = 0; u < NP; ++u)
#pragma unroll
                for (int k = 0; k < D / 32; ++k)
                    mma_f8(tmem + pipe * 128 + half * kPass, gemm::smem_desc(qb + u * S::kCodes + 32 * k, D),
                           gemm::smem_desc(kb + 32 * k, D), scores_desc<kE5M2>(), u > 0 || k > 0);
            gemm::mma_commit(bar(B_SFULL + 2 * pipe + half));
            if (half == 1) {
                gemm::mma_commit(bar(B_KEMPTY + stage));
                if (!kTwo && last && pipe == 0) gemm::mma_commit(bar(B_QDONE));
            }
            return true;
        };
        auto products = [&](int t, int half, bool started) {
            const int stage = (n + t) & 1;
            if (half == 0 &&
                !tile_wait(p, bar(B_HFULL + stage), ((n + t) >> 1) & 1, &sh_abort))
                return false;
            gemm::tmem_fence_after();
            const uint32_t vb = sbase + S::kVh + stage * S::kHalf + half * (kPass / 16 * 2048);
#pragma unroll
            for (int k = 0; k < kPass / 16; ++k)
                mma_f16_ts(tmem + kTmemO + pipe * 128, tmem + pipe * 128 + half * kPass + 8 * k,
                           value_desc(vb + k * 2048), products_desc<D>(), started || k > 0);
            if (half == 1) gemm::mma_commit(bar(B_HEMPTY + stage));
            gemm::mma_commit(bar(B_ODONE + 2 * pipe + half));
            return true;
        };
        auto segments = [&]() {
#pragma unroll 1
            while (walk.next(p, kRows)) {
                const int T = walk.t1 - walk.t0;
                if (!tile_wait(p, bar(B_QREADY + (kTwo ? pipe : 0)), segment & 1, &sh_abort))
                    return;
                const int first = kTwo ? 0 : pipe;
                if (first < T)
#pragma unroll 1
                    for (int half = 0; half < 2; ++half)
                        if (!scores(first, half, first + kEach >= T)) return;
#pragma unroll 1
                for (int t = first; t < T; t += kEach, ++items) {
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        if (!tile_wait(p, bar(B_PFULL + 2 * pipe + half), items & 1, &sh_abort) ||
                            !products(t, half, t > first || half > 0))
                            return;
                        if (t + kEach < T && !scores(t + kEach, half, t + 2 * kEach >= T)) return;
                    }
                }
                if (!kTwo && pipe == 1) {
                    gemm::mbar_arrive(bar(B_NEXT));
                    if (!tile_wait(p, bar(B_NEXT), segment & 1, &sh_abort)) return;
                }
                n += T;
                ++segment;
            }
        };
        if (lane == 0) {
            segments();
            // nothing may be in flight when the tensor memory goes
            gemm::mma_commit(bar(B_DRAIN));
            const unsigned long long t0 = gemm::now_ns();
            while (!gemm::mbar_try_wait(bar(B_DRAIN), 0))
                if (gemm::now_ns() - t0 > kWaitLimitNs) break;
        }
        __syncwarp();
    } else if (warp >= kSoftWarps) {
        // ---------------- values to binary16 ----------------
        Walk walk;
        walk.begin(cur);
        const int cw = warp - kSoftWarps;
        constexpr int kPer = D / 16;         // 16-code chunks of a row
        constexpr int kLoads = kPer;         // of 32 rows by 32 lanes
        int vs = 0;
        uint32_t vp = 0;
        int n = 0;
        bool alive = true;
#pragma unroll 1
        while (alive && walk.next(p, kRows)) {
#pragma unroll 1
            for (int t = walk.t0; t < walk.t1; ++t, ++n) {
                const uint32_t ti =
                    sbase + S::kInfo + (n & (kInfos - 1)) * (uint32_t)sizeof(TileInfo);
                const int stage = n & 1;
                alive = tile_wait(p, bar(B_INFO + (n & (kInfos - 1))), (n >> 3) & 1, &sh_abort) &&
                        tile_wait(p, bar(B_VFULL + vs), vp, &sh_abort) &&
                        tile_wait(p, bar(B_HEMPTY + stage), ((n >> 1) & 1) ^ 1, &sh_abort);
                alive = __all_sync(0xffffffffu, alive);
                if (!alive) break;
                const uint32_t from = sbase + S::kV + vs * S::kCodes,
                               to = sbase + S::kVh + stage * S::kHalf;
                const uint32_t ok = __float_as_uint(lds_f(ti + kInfoOk + 4 * cw));
                // Behind the context a value may be hidden from some rows, and
                // 0 times NaN or infinity would reach them: such elements
                // become zero here and are added at the end to the rows that
                // see them.  The context's own reach every row as they are.
                const bool past = (t + 1) * kTileKeys > walk.sg.s.ctx;
                const int hideable = walk.sg.s.ctx - t * kTileKeys;  // rows from here on
                bool any = false;
#pragma unroll 1
                for (int i = 0; i < kLoads; ++i) {
                    // eight neighbouring lanes store two rows' neighbouring
                    // chunks, which the swizzle keeps in different banks
                    const int r = D == 128 ? ((lane >> 2) & 3) + 4 * i : (lane >> 2) + 8 * i;
                    const int x = D == 128 ? (lane & 3) | ((lane >> 4) << 2) : lane & 3;
                    const int row = cw * 32 + r;
                    uint4 c = gemm::lds128(from + code_at<D>(row, x));
                    if (!((ok >> r) & 1u)) c = make_uint4(0, 0, 0, 0);
                    if (past && row >= hideable) {
                        const uint4 f = make_uint4(finite_codes<kE5M2>(c.x), finite_codes<kE5M2>(c.y),
                                                   finite_codes<kE5M2>(c.z), finite_codes<kE5M2>(c.w));
                        any |= c.x != f.x || c.y != f.y || c.z != f.z || c.w != f.w;
                        c = f;
                    }
                    uint32_t h[8];
                    kv::codes4_to_h2<kE5M2>(c.x, h[0], h[1]);
                    kv::codes4_to_h2<kE5M2>(c.y, h[2], h[3]);
                    kv::codes4_to_h2<kE5M2>(c.z, h[4], h[5]);
                    kv::codes4_to_h2<kE5M2>(c.w, h[6], h[7]);
                    gemm::sts128(to + half_at(row, x >> 2, (x & 3) * 2),
                                 make_uint4(h[0], h[1], h[2], h[3]));
                    gemm::sts128(to + half_at(row, x >> 2, (x & 3) * 2 + 1),
                                 make_uint4(h[4], h[5], h[6], h[7]));
                }
                if (any) sh_nonfinite = 1;
                gemm::fence_async_shared();
                __syncwarp();
                if (lane == 0) {
                    gemm::mbar_arrive(bar(B_VEMPTY + vs));
                    gemm::mbar_arrive(bar(B_HFULL + stage));
                }
                if (++vs == S::kStagesV) {
                    vs = 0;
                    vp ^= 1;
                }
            }
        }
    } else {
        // ---------------- softmax ----------------
        Walk &walk = sh_walk[warp];
        if (lane == 0) walk.begin(cur);
        const int pipe = warp >> 2;
        const int r = threadIdx.x & 127;  // row of the pipeline = lane of tensor memory
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes
        const uint32_t ts = tmem + pipe * 128 + lanes, to = tmem + kTmemO + pipe * 128 + lanes;
        int n = 0;                            // tiles of finished segments
        int items = 0, segment = 0, merges = 0;  // items: passes of this pipeline
        bool alive = true;
        auto wait = [&](int b, int parity) {
            alive = tile_wait(p, bar(b), parity & 1, &sh_abort);
            alive = __all_sync(0xffffffffu, alive);
            return alive;
        };
        while (alive) {
            __syncwarp();
            int go = 0;
            if (lane == 0) go = walk.next(p, kRows);
            if (!__shfl_sync(0xffffffffu, go, 0)) break;
            __syncwarp();
            const Segment &sg = walk.sg;
            const int T = walk.t1 - walk.t0;
            const int R = sg.block * kRows + (kTwo ? pipe * kTileRows : 0) + r;
            const int tok = R / p.G, hq = sg.head * p.G + (R - tok * p.G);
            const bool live = tok < sg.s.n;
            const bool warp_live = __any_sync(0xffffffffu, live);
            if (kTwo || pipe == 0) {
                // Q's e4m3 pieces, each row scaled by a power of two that
                // brings its largest magnitude to [128, 256): piece u is the
                // rounded rest.  What is under 2^-17 of the row's largest is
                // lost.  A row that is not finite becomes NaN.  D / 8 lanes
                // read a row, four loads at a time.
                constexpr int kLanes = D / 8, kSide = 32 / kLanes, kN = 32 / kSide, kB = 4;
                const uint16_t *src = static_cast<const uint16_t *>(p.q.data);
                const int64_t own =
                    live ? (sg.row0 + tok) * p.q.ts + (int64_t)hq * p.q.hs : -1;
                const int chunk = lane % kLanes, side = lane / kLanes;
                const uint32_t inf = NP == 2 ? 0x7f80u : 0x7c00u;
                const uint32_t qb = sbase + S::kQ + (kTwo ? pipe * NP * S::kCodes : 0);
                auto load = [&](int i, uint4 (&w)[kB]) {
#pragma unroll
                    for (int u = 0; u < kB; ++u) {
                        const int64_t at =
                            __shfl_sync(0xffffffffu, own, (i + u) * kSide + side);
                        w[u] = make_uint4(0, 0, 0, 0);
                        if (at >= 0) w[u] = ld_stream(src + at + chunk * 8);
                    }
                };
                uint4 w[kB], ahead[kB];
                load(0, ahead);
#pragma unroll 1
                for (int i = 0; i < kN; i += kB) {
#pragma unroll
                    for (int u = 0; u < kB; ++u) w[u] = ahead[u];
                    if (i + kB < kN) load(i + kB, ahead);
#pragma unroll
                    for (int u = 0; u < kB; ++u) {
                        const int r = (warp & 3) * 32 + (i + u) * kSide + side;
                        // the row's largest magnitude, as the integer it sorts as
                        const uint32_t m2 =
                            __vmaxu2(__vmaxu2(w[u].x & 0x7fff7fffu, w[u].y & 0x7fff7fffu),
                                     __vmaxu2(w[u].z & 0x7fff7fffu, w[u].w & 0x7fff7fffu));
                        uint32_t most = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
                        for (int x = kLanes / 2; x > 0; x >>= 1)
                            most = max(most, __shfl_xor_sync(0xffffffffu, most, x));
                        const float amax = NP == 2 ? __uint_as_float(most << 16)
                                                   : DT<__half>::w2f(most).x;
                        const bool finite = most < inf;
                        int ex = finite && amax > 0.f ? (int)(__float_as_uint(amax) >> 23) - 127 : 7;
                        ex = max(ex, -100);
                        const float by = power_of_two(7 - ex);
                        if (chunk == 0) sh_back[(kTwo ? pipe * kTileRows : 0) + r] = power_of_two(ex - 7);
                        float f[8];
                        if (NP == 2) DT<__nv_bfloat16>::unpack(w[u], f);
                        else DT<__half>::unpack(w[u], f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] *= by;
                        const uint32_t to = qb + code_at<D>(r, chunk >> 1) + 8 * (chunk & 1);
#pragma unroll
                        for (int v = 0; v < NP; ++v) {
                            uint32_t c[2];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                c[h] = fp8x2(f[4 * h], f[4 * h + 1], Q_E4M3) |
                                       fp8x2(f[4 * h + 2], f[4 * h + 3], Q_E4M3) << 16;
                                uint32_t lo, hi;
                                kv::codes4_to_h2<false>(c[h], lo, hi);
                                const float2 a = DT<__half>::w2f(lo), b = DT<__half>::w2f(hi);
                                f[4 * h] -= a.x;
                                f[4 * h + 1] -= a.y;
                                f[4 * h + 2] -= b.x;
                                f[4 * h + 3] -= b.y;
                                if (!finite) c[h] = 0x7f7f7f7fu;
                            }
                            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(
                                             to + v * S::kCodes),
                                         "r"(c[0]), "r"(c[1])
                                         : "memory");
                        }
                    }
                }
                gemm::fence_async_shared();
                __syncwarp();
                if (lane == 0) gemm::mbar_arrive(bar(B_QREADY + (kTwo ? pipe : 0)));
            }

            RowLane row;
            row.off = 0.f;
            row.set = !live;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                row.sub[i] = 0.f;
                row.l[i] = two(0.f, 0.f);
            }
            bool done = false;  // products of this segment are issued
            constexpr int kEach = kTwo ? 1 : 2;
            const int t_first = kTwo ? 0 : pipe;
            if (!wait(B_QREADY + (kTwo ? pipe : 0), segment)) break;
            const float back = sh_back[(kTwo ? pipe * kTileRows : 0) + r];
            rows_from_owner(back, row.back);
            for (int t = t_first; t < T; t += kEach) {
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    if (!wait(B_SFULL + 2 * pipe + half, items >> 1)) break;
                    if (!wait(B_INFO + ((n + t) & (kInfos - 1)), (n + t) >> 3)) break;
                    gemm::tmem_fence_after();
                    const uint32_t info = sbase + S::kInfo +
                                          ((n + t) & (kInfos - 1)) * (uint32_t)sizeof(TileInfo);
                    const uint32_t ti = info + 4 * kPass * half, tsh = ts + kPass * half;
                    const int j0 = (walk.t0 + t) * kTileKeys + kPass * half;
                    const uint64_t okw = lds64(info + kInfoOk + 8 * half);
                    uint32_t v0 = (uint32_t)okw, v1 = (uint32_t)(okw >> 32);
                    const bool edge = okw != ~0ull || j0 + kPass > sg.s.ctx;  // uniform
                    if (edge) {
                        const int d0 = j0 - sg.s.ctx;  // drafted token of v0's bit 0
                        v0 &= live ? seen_word(p, sg.row0 + tok, tok, d0) : 0u;
                        v1 &= live ? seen_word(p, sg.row0 + tok, tok, d0 + 32) : 0u;
                    }
                    // a warp without rows leaves its weights as they are: they
                    // reach no other row
                    if (warp_live) {
                        float lift = lds_f(info + kInfoLift + 4 * half);
                        if (edge && lds_f(info + kInfoWide + 4 * half) != 0.f)
                            lift = row_lift(ti, v0, v1);
                        if (!__all_sync(0xffffffffu, row.set)) {
                            const float top = edge ? row_top<true>(tsh, ti, v0, v1, back)
                                                   : row_top<false>(tsh, ti, 0, 0, back);
                            if (!row.set && top > -INFINITY) {
                                row.off = first_offset(top, kCentre - lift);
                                row.set = true;
                            }
                            rows_from_owner(-row.off, row.sub);
                        }
                        auto settled = [&]() {
                            const bool in = wait(B_ODONE + 2 * pipe + (half ^ 1), (items - 1) >> 1);
                            gemm::tmem_fence_after();
                            return in;
                        };
                        if (edge)
                            alive = row_weights<D, true>(tsh, to, done, ti, v0, v1, lift, row,
                                                         settled);
                        else
                            alive = row_weights<D, false>(tsh, to, done, ti, v0, v1, lift, row,
                                                          settled);
                    }
                    tmem_st_wait();
                    gemm::tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) gemm::mbar_arrive(bar(B_PFULL + 2 * pipe + half));
                    if (!alive) break;
                    ++items;
                    done = true;
                }
                if (!alive) break;
            }
            if (!alive) break;
            if (done) {
                if (!wait(B_ODONE + 2 * pipe + 1, (items - 1) >> 1)) break;
                gemm::tmem_fence_after();
            }
            float row_l = row_sum(row);
            const bool whole = walk.t0 == 0 && walk.t1 == sg.s.tiles;
            float *buf = reinterpret_cast<float *>(smem + S::kQ);  // [column][row]
            const bool joined = !kTwo && T > 1;
            if (joined && pipe == 1) {
                // this pipeline's state, over the queries once the other
                // pipeline's last scores are done as well
                if (!wait(B_QDONE, segment)) break;
                sh_ml[r] = make_float2(row_l, row.off);
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    gemm::tmem_ld32(to + 32 * c, o);
#pragma unroll
                    for (int j = 0; j < 32; ++j) buf[(32 * c + j) * kTileRows + r] = o[j];
                }
                __syncwarp();
                if (lane == 0) gemm::mbar_arrive(bar(B_MERGE));
            } else if (kTwo || pipe == 0) {
                float f0 = 1.f, f1 = 0.f;
                if (joined) {
                    if (!wait(B_MERGE, merges)) break;
                    ++merges;
                    // both in the units of the larger offset
                    const float2 o1 = sh_ml[r];
                    const float oo = fmaxf(row_l == 0.f ? -INFINITY : row.off,
                                           o1.x == 0.f ? -INFINITY : o1.y);
                    f0 = row_l == 0.f ? 0.f : row.off == oo ? 1.f : exp2_fast(row.off - oo);
                    f1 = o1.x == 0.f ? 0.f : o1.y == oo ? 1.f : exp2_fast(o1.y - oo);
                    row_l = row_l * f0 + o1.x * f1;
                    row.off = oo;
                }
                const int64_t slot = 2 * (int64_t)blockIdx.x + (walk.t0 == 0 ? 1 : 0);
                const int64_t prow = slot * kRows + (kTwo ? pipe * kTileRows : 0) + r;
                const float by = !whole ? 1.f : row_l == 0.f ? 0.f : 1.f / row_l;
                if (!whole)
                    p.ml[prow] = make_float2(row_l == 0.f ? -INFINITY : row.off, row_l);
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    if (done) gemm::tmem_ld32(to + 32 * c, o);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        // (a factor of zero too: it keeps a NaN)
                        float v = done ? o[j] * f0 : 0.f;
                        if (joined) v += buf[(32 * c + j) * kTileRows + r] * f1;
                        o[j] = v * by;
                    }
                    if (sh_nonfinite && live)
                        add_nonfinite<kE5M2>(p, sg, tok, walk.t0 * kTileKeys, walk.t1 * kTileKeys,
                                             32 * c, o);
                    if (whole) {
                        if (live) {
#pragma unroll
                            for (int j = 0; j < 32; j += 4)
                                store_out4(p, sg.row0 + tok, hq, 32 * c + j,
                                           make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            const float v8[8] = {o[j], o[j + 1], o[j + 2], o[j + 3],
                                                 o[j + 4], o[j + 5], o[j + 6], o[j + 7]};
                            st_global32f(p.part + prow * D + 32 * c + j, v8);
                        }
                    }
                }
                if (walk.t0 == 0 && pipe == 0 && r == 0)
                    p.joins[walk.seg0 + walk.which] =
                        Join{(int)blockIdx.x,
                             whole ? -1 : part_of(sh_cur.each, sh_cur.more, walk.last_unit),
                             (int)sg.row0, sg.s.n, sg.head, sg.block, 0, 0};
            }
            gemm::tmem_fence_before();  // O is read before the next segment's products
            if (!kTwo) {
                // The pipelines begin a segment together: the next queries go
                // where the joined state was read, and who skipped segments of
                // a single tile could take an old phase of a barrier for its
                // own.
                __syncwarp();
                if (lane == 0) gemm::mbar_arrive(bar(B_NEXT));
                if (!wait(B_NEXT, segment)) break;
            }
            n += T;
            ++segment;
        }
    }
    gemm::tmem_fence_before();
    __syncthreads();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
    if (sh_abort) give_up(p, sh_cur, kRows);  // last: its lanes part
}

}  // namespace tree
}  // namespace rarn
