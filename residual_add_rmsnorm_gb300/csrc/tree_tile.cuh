// tree_tile.cuh -- the attention of tree_attn.cuh for many rows per key head:
// 128 or 256 rows (drafted tokens x query heads of a group) against tiles of
// 128 keys on the fifth-generation tensor cores.
//
//   S = Q K^T, P = 2^(s - m) vs, O = P V      binary16 operands, binary32 sums
//
// With more than a few dozen rows the second product's conversions no longer
// hide behind the reads, and mma.sync's binary16 rate (a quarter of
// tcgen05's) becomes the bound; here the codes become binary16 once per tile
// in shared memory, whatever the number of rows.
//
// One CTA per SM, persistent over its part of the line of tiles:
//   * eight converter warps load two tiles ahead into registers, convert the
//     codes (exactly) and store keys and values in 128-byte-swizzled rows,
//     and the tile's scales beside them;
//   * two pipelines of four softmax warps, a thread per row: scores from
//     tensor memory, running maximum with slack, weights rounded to binary16
//     over the scores' columns; one thread of each issues its tcgen05.mma: S
//     into the pipeline's 128 columns, and O += P V with P read from tensor
//     memory and V from the same row layout as K (as the N-major operand).
// Sixteen warps in all: with a seventeenth for the products a thread has 96
// registers instead of 128, and what spills goes through the little L1 that
// shared memory leaves (three times the time).
// With up to 128 rows the pipelines take alternate tiles of the same rows, and
// their states are joined at the end; with up to 256 rows each has its own
// 128. While one pipeline is at its softmax the other's products run.
//
// Every wait is bounded; one that runs out sets watchdog bit 5, the CTA's
// warps give up together, and its tensor memory is freed.
#pragma once

#include "tree_attn.cuh"

namespace rarn {
namespace tree {

constexpr int kTileKeys = 128;   // keys of a tile
constexpr int kTileRows = 128;   // rows of a pipeline
constexpr int kSoftWarps = 8;
constexpr int kConvWarps = 8;       // 16 keys of a tile each
constexpr int kTileThreads = 32 * (kSoftWarps + kConvWarps);
constexpr int kMaxTileCtas = 160;

// What the softmax needs of a tile besides its scores.
struct TileInfo {
    float kk[kTileKeys];      // key scale x softmax scale x what undoes Q's scaling
    float vs[kTileKeys];      // value scale, 0 where there is no key
    float vmax[kConvWarps];   // largest finite |vs| of 16 keys
    uint16_t ok[kConvWarps];  // keys that exist
};

template <int D>
struct TileSmem {
    static constexpr int kOperand = kTileKeys * D * 2;  // one tile of K, V or Q in binary16
    static constexpr int kQ = 0;                        // two of them
    static constexpr int kK = 2 * kOperand;             // two stages
    static constexpr int kV = 4 * kOperand;             // two stages
    static constexpr int kInfo = 6 * kOperand;          // four tiles
    static constexpr int kBytes = kInfo + 4 * (int)sizeof(TileInfo) + 1024;
};

// Barriers, in one array.
enum Bar : int {
    B_KFULL = 0, B_KEMPTY = 2, B_VFULL = 4, B_VEMPTY = 6, B_SFULL = 8, B_PFULL = 10, B_ODONE = 12,
    B_INFO = 14, B_QMAX = 18, B_QREADY = 19, B_MERGE = 20, B_DRAIN = 21, B_QDONE = 22, B_NEXT = 23,
    B_COUNT = 24
};

// A CTA's share of the line, segment by segment.  Every role walks it alike.
struct Walk {
    const Params &p;
    int rows;
    int at, hi, base, seg0;
    Segment sg;
    int t0, t1, which;

    __device__ __forceinline__ Walk(const Params &p_, int rows_, const Cursor &c)
        : p(p_), rows(rows_), at(c.lo), hi(c.hi), base(c.base), seg0(c.seg0), t0(0), t1(0),
          which(0) {
        sg.b = c.b;
    }
    // The next segment; false when there is none.
    __device__ __forceinline__ bool next() {
        at += t1 - t0;
        t0 = t1 = 0;
        while (at < hi) {
            sg.s = seq_of(p, sg.b, rows, kTileKeys);
            const int units = (int)units_of(p, sg.s);
            if (at < base + units) {
                const int rel = at - base;
                which = (unsigned)rel / (unsigned)sg.s.tiles;
                t0 = rel - which * sg.s.tiles;
                t1 = min(t0 + hi - at, sg.s.tiles);
                sg.head = (unsigned)which / (unsigned)sg.s.blocks;
                sg.block = which - sg.head * sg.s.blocks;
                sg.row0 = p.starts[sg.b];
                return true;
            }
            base += units;
            seg0 += p.cache.heads * sg.s.blocks;
            ++sg.b;
        }
        return false;
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
            } else if (t - t0 > kWaitLimitNs) {
                *abort_flag = 1;
                atomicOr(p.watchdog, kWatchTree);
                return false;
            }
        }
    }
}

// Exponent of a block's largest query magnitude (binary32 bits): Q is scaled
// by 2^(13 - e), its largest element then in [2^13, 2^14).
__device__ __forceinline__ int query_exponent(unsigned int amax) {
    const int e = amax ? (int)(amax >> 23) - 127 : 13;
    return e < -100 ? -100 : e;
}

__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }

// Codes that are NaN or infinite become zero.
template <bool kE5M2>
__device__ __forceinline__ uint32_t finite_codes(uint32_t w) {
    constexpr uint32_t top = kE5M2 ? 0x7c7c7c7cu : 0x7f7f7f7fu;
    return w & ~__vcmpeq4(w & top, top);
}

// Byte of 16-byte chunk c (8 elements) of a row of `half` 64 elements: K-major
// rows for Q and K, and the N-major form of V, are one layout.
template <int D>
__device__ __forceinline__ uint32_t operand_at(int row, int half, int c) {
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

template <int N, bool kNMajorB>
__host__ __device__ constexpr uint32_t tile_desc() {
    return gemm::instr_desc<__half, N>() | (kNMajorB ? 1u << 16 : 0u);
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
__device__ __forceinline__ uint32_t seen_word(const Params &p, int64_t row, int tok, int n,
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
    (void)n;
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

// 16 columns of tensor memory on their way to registers, and their arrival.
__device__ __forceinline__ void tmem_ld16_begin(uint32_t taddr, float (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
          "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]),
          "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld16_end(float (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]),
                   "+f"(r[6]), "+f"(r[7]), "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]),
                   "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}

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

// A row's largest score of a tile: columns of S at `ts` times the keys'
// factors.  kEdge: only where bits of vis are set.
template <bool kEdge>
__device__ __forceinline__ float row_top(uint32_t ts, const TileInfo &ti,
                                         const uint32_t (&vis)[4]) {
    float t0 = -INFINITY, t1 = -INFINITY;
    float buf[2][16];
    tmem_ld16_begin(ts, buf[0]);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        float(&s)[16] = buf[c & 1];
        tmem_ld16_end(s);
        if (c < 7) tmem_ld16_begin(ts + 16 * (c + 1), buf[(c + 1) & 1]);
        const uint32_t v16 = kEdge ? vis[c >> 1] >> (16 * (c & 1)) : 0u;
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const ulonglong2 kk = *reinterpret_cast<const ulonglong2 *>(ti.kk + 16 * c + j);
            float2 a = apart(mul2(two(s[j], s[j + 1]), kk.x));
            float2 b = apart(mul2(two(s[j + 2], s[j + 3]), kk.y));
            if (kEdge) {
                if (!((v16 >> j) & 1u)) a.x = -INFINITY;
                if (!((v16 >> (j + 1)) & 1u)) a.y = -INFINITY;
                if (!((v16 >> (j + 2)) & 1u)) b.x = -INFINITY;
                if (!((v16 >> (j + 3)) & 1u)) b.y = -INFINITY;
            }
            t0 = max3(t0, a.x, a.y);
            t1 = max3(t1, b.x, b.y);
        }
    }
    return fmaxf(t0, t1);
}

// A row's weights of a tile, 2^(score - off) times the value scales, in
// binary16 over the scores' columns; returns the sum of 2^(score - off).
template <bool kEdge>
__device__ __forceinline__ float row_weights(uint32_t ts, const TileInfo &ti,
                                             const uint32_t (&vis)[4], float off) {
    uint64_t l0 = two(0.f, 0.f), l1 = l0;
    const uint64_t shift = two(-off, -off);
    float buf[2][16];
    tmem_ld16_begin(ts, buf[0]);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        float(&s)[16] = buf[c & 1];
        tmem_ld16_end(s);
        if (c < 7) tmem_ld16_begin(ts + 16 * (c + 1), buf[(c + 1) & 1]);
        const uint32_t v16 = kEdge ? vis[c >> 1] >> (16 * (c & 1)) : 0u;
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const ulonglong2 kk = *reinterpret_cast<const ulonglong2 *>(ti.kk + 16 * c + j);
            const ulonglong2 vs = *reinterpret_cast<const ulonglong2 *>(ti.vs + 16 * c + j);
            float2 a = apart(fma2(two(s[j], s[j + 1]), kk.x, shift));
            float2 b = apart(fma2(two(s[j + 2], s[j + 3]), kk.y, shift));
            const uint32_t v4 = v16 >> j;
            if (kEdge) {
                if (!(v4 & 1u)) a.x = -INFINITY;
                if (!(v4 & 2u)) a.y = -INFINITY;
                if (!(v4 & 4u)) b.x = -INFINITY;
                if (!(v4 & 8u)) b.y = -INFINITY;
            }
            const uint64_t pa = two(exp2_fast(a.x), exp2_fast(a.y));
            const uint64_t pb = two(exp2_fast(b.x), exp2_fast(b.y));
            l0 = add2(l0, pa);
            l1 = add2(l1, pb);
            a = apart(mul2(pa, vs.x));
            b = apart(mul2(pb, vs.y));
            if (kEdge) {
                if (!(v4 & 1u)) a.x = 0.f;
                if (!(v4 & 2u)) a.y = 0.f;
                if (!(v4 & 4u)) b.x = 0.f;
                if (!(v4 & 8u)) b.y = 0.f;
            }
            w[j / 2] = pack_h2(a.x, a.y);
            w[j / 2 + 1] = pack_h2(b.x, b.y);
        }
        tmem_st8(ts + 8 * c, w);  // behind every load that is under way
    }
    const float2 x = apart(add2(l0, l1));
    return x.x + x.y;
}

// The k of an offset m - k.
__device__ __forceinline__ int k_of(float off, float m) {
    return __float2int_rn((m == -INFINITY ? 0.f : m) - off);
}

// ---------------------------------------------------------------------------
// Converters
// ---------------------------------------------------------------------------

// A tile as a converter lane knows it: key (lane & 15) of the warp's 16.
struct Look {
    int64_t code;     // where the key's codes lie, < 0: nowhere
    float sc;         // lanes 0 .. 15: its key scale, 16 .. 31: its value scale
    bool past;        // the tile reaches behind the context
    bool first;       // of its segment
};

// Loads of each of K and V by a converter thread: 256 threads, 16 codes a load.
template <int D>
constexpr int kConvLoads = D / 32;

// Where a converter thread's i-th load belongs: row of the warp's 16, chunk of
// 16 codes.  Eight neighbouring lanes store two rows' neighbouring chunks,
// which the swizzle keeps in different banks.
template <int D>
__device__ __forceinline__ void conv_place(int lane, int i, int &row, int &x) {
    if constexpr (D == 128) {
        row = ((lane >> 2) & 3) + 4 * i;
        x = (lane & 3) | ((lane >> 4) << 2);
    } else {
        row = (lane >> 2) + 8 * i;
        x = lane & 3;
    }
}

__device__ __forceinline__ uint4 ld_past_l1(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// A converter thread's share of a tile's codes.
template <int D>
struct Codes {
    uint4 k[kConvLoads<D>], v[kConvLoads<D>];

    __device__ __forceinline__ void load(const Cache &c, int64_t code) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < kConvLoads<D>; ++i) {
            int row, x;
            conv_place<D>(lane, i, row, x);
            const int64_t at = __shfl_sync(0xffffffffu, code, row);
            k[i] = v[i] = make_uint4(0, 0, 0, 0);
            if (at >= 0) {
                k[i] = ld_past_l1(c.k + at + x * 16);
                v[i] = ld_past_l1(c.v + at + x * 16);
            }
        }
    }
};

// 16 codes to binary16 into a tile of an operand.
template <int D, bool kE5M2>
__device__ __forceinline__ void store_codes(uint32_t base, int row, int x, const uint4 &c) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t h[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) kv::codes4_to_h2<kE5M2>(w[j], h[2 * j], h[2 * j + 1]);
    const int half = x >> 2, ch = (x & 3) * 2;
    gemm::sts128(base + operand_at<D>(row, half, ch), make_uint4(h[0], h[1], h[2], h[3]));
    gemm::sts128(base + operand_at<D>(row, half, ch + 1), make_uint4(h[4], h[5], h[6], h[7]));
}

// ---------------------------------------------------------------------------

// kTwo: 256 rows, 128 to each pipeline; else 128, tiles alternate.
template <int D, bool kE5M2, bool kTwo>
__global__ void __launch_bounds__(kTileThreads, 1) k_tree_tile(const Params p) {
    using S = TileSmem<D>;
    constexpr int kRows = kTwo ? 2 * kTileRows : kTileRows;
    constexpr uint32_t kTmemO = 256;  // O of pipeline 0; S are columns 0 and 128
    extern __shared__ uint8_t smem_raw[];
    __shared__ int64_t sh_part[16];
    __shared__ __align__(8) uint64_t sh_bar[B_COUNT];
    __shared__ uint32_t sh_tmem;
    __shared__ volatile int sh_abort;
    __shared__ volatile int sh_nonfinite;  // a value was kept out of the products
    __shared__ unsigned int sh_amax[2];    // of the block's queries, by segment parity
    __shared__ float2 sh_ml[kTileRows];  // pipeline 1's l and offset
    __shared__ float sh_m[kTileRows];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    TileInfo *info = reinterpret_cast<TileInfo *>(smem + S::kInfo);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t bars = smem_u32(sh_bar);
    auto bar = [&](int b) { return bars + 8 * b; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            gemm::mbar_init(bar(B_KFULL + i), kConvWarps);
            gemm::mbar_init(bar(B_KEMPTY + i), kTwo ? 2 : 1);
            gemm::mbar_init(bar(B_VFULL + i), kConvWarps);
            gemm::mbar_init(bar(B_VEMPTY + i), kTwo ? 2 : 1);
            gemm::mbar_init(bar(B_SFULL + i), 1);
            gemm::mbar_init(bar(B_PFULL + i), 4);
            gemm::mbar_init(bar(B_ODONE + i), 1);
        }
        for (int i = 0; i < 4; ++i) gemm::mbar_init(bar(B_INFO + i), kConvWarps);
        gemm::mbar_init(bar(B_QMAX), kTwo ? 8 : 4);
        gemm::mbar_init(bar(B_QREADY), kTwo ? 8 : 4);
        gemm::mbar_init(bar(B_MERGE), 4);
        gemm::mbar_init(bar(B_DRAIN), 2);
        gemm::mbar_init(bar(B_QDONE), 1);
        gemm::mbar_init(bar(B_NEXT), 4);
        gemm::fence_async_shared();
        sh_abort = 0;
        sh_nonfinite = 0;
        sh_amax[0] = sh_amax[1] = 0;
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
    Walk walk(p, kRows, cur);

    if (warp >= kSoftWarps) {
        // ---------------- converters ----------------
        const int cw = warp - kSoftWarps;
        // The stream of tiles over all segments.  While tile n is converted,
        // the codes of n + 1 and n + 2 are on their way and the pages of
        // n + 3 are looked up.
        int tile = 0;
        bool more = walk.next();
        if (more) tile = walk.t0;
        struct Ahead {
            int j, head;
            int page;    // -1: none, -2: behind the sequence
            bool past, first, there;
        } ah;
        auto look_up = [&]() {  // begins the look-up of the stream's next tile
            ah.there = more;
            if (!more) return;
            const Segment &sg = walk.sg;
            ah.j = tile * kTileKeys + cw * 16 + (lane & 15);
            ah.head = sg.head;
            ah.past = (tile + 1) * kTileKeys > sg.s.ctx;
            ah.first = tile == walk.t0;
            ah.page = -2;
            if (ah.j < sg.s.len) ah.page = max(-1, p.table[sg.b * p.table_stride + p.page_of(ah.j)]);
            if (++tile >= walk.t1) {
                more = walk.next();
                tile = walk.t0;
            }
        };
        auto found = [&](Look &x) {  // ends it
            x.code = -1;
            x.sc = 0.f;
            if (!ah.there) return false;
            x.past = ah.past;
            x.first = ah.first;
            if (ah.page >= 0 && ah.page < p.cache.pages) {
                const KeyAt at = place(p, ah.page, p.offset_in_page(ah.j), ah.head);
                x.code = at.code;
                x.sc = (lane < 16 ? p.cache.k_scale : p.cache.v_scale)[at.scale];
            } else if (ah.page != -2) {
                atomicOr(p.watchdog, kv::kWatchIndex);
            }
            return true;
        };
        int segments = 0;  // begun by the tiles stored
        int n = 0;         // tiles stored
        bool alive = true;
        auto store = [&](Codes<D> &c, const Look &now) {
            const int stage = n & 1;
            const uint32_t parity = ((n >> 1) & 1) ^ 1;
            TileInfo &ti = info[n & 3];
            const uint32_t kbase = sbase + S::kK + stage * S::kOperand;
            const uint32_t vbase = sbase + S::kV + stage * S::kOperand;
            alive = tile_wait(p, bar(B_KEMPTY + stage), parity, &sh_abort);
            if (now.first) {
                // the scaling of this segment's queries goes into the key scales
                alive = alive && tile_wait(p, bar(B_QREADY), segments & 1, &sh_abort);
                ++segments;
            }
            alive = __all_sync(0xffffffffu, alive);
            if (!alive) return;
#pragma unroll
            for (int i = 0; i < kConvLoads<D>; ++i) {
                int row, ch;
                conv_place<D>(lane, i, row, ch);
                store_codes<D, kE5M2>(kbase, cw * 16 + row, ch, c.k[i]);
            }
            const float undo =
                power_of_two(query_exponent(sh_amax[(segments - 1) & 1]) - 13) * p.scale_log2;
            const float vabs = fabsf(now.sc);
            const float vmax = warp_max(lane >= 16 && vabs < INFINITY ? vabs : 0.f);
            const uint32_t ok = __ballot_sync(0xffffffffu, now.code >= 0);
            if (lane < 16) ti.kk[cw * 16 + lane] = now.sc * undo;
            else ti.vs[cw * 16 + lane - 16] = now.sc;
            if (lane == 0) {
                ti.vmax[cw] = vmax;
                ti.ok[cw] = (uint16_t)ok;
            }
            // Behind the context a value may be hidden from some rows, and 0
            // times NaN or infinity would reach them: such elements become
            // zero here and are added at the end to the rows that see them.
            if (now.past) {
                bool any = false;
#pragma unroll
                for (int i = 0; i < kConvLoads<D>; ++i) {
                    const uint4 w = c.v[i];
                    c.v[i] = make_uint4(finite_codes<kE5M2>(w.x), finite_codes<kE5M2>(w.y),
                                        finite_codes<kE5M2>(w.z), finite_codes<kE5M2>(w.w));
                    any |= w.x != c.v[i].x || w.y != c.v[i].y || w.z != c.v[i].z ||
                           w.w != c.v[i].w;
                }
                if (any) sh_nonfinite = 1;
            }
            gemm::fence_async_shared();
            __syncwarp();
            if (lane == 0) {
                gemm::mbar_arrive(bar(B_KFULL + stage));
                gemm::mbar_arrive(bar(B_INFO + (n & 3)));
            }
            alive = tile_wait(p, bar(B_VEMPTY + stage), parity, &sh_abort);
            alive = __all_sync(0xffffffffu, alive);
            if (!alive) return;
#pragma unroll
            for (int i = 0; i < kConvLoads<D>; ++i) {
                int row, ch;
                conv_place<D>(lane, i, row, ch);
                store_codes<D, kE5M2>(vbase, cw * 16 + row, ch, c.v[i]);
            }
            gemm::fence_async_shared();
            __syncwarp();
            if (lane == 0) gemm::mbar_arrive(bar(B_VFULL + stage));
            ++n;
        };
        // looks of tiles n, n + 1 and n + 2; codes of n and n + 1
        Codes<D> c0, c1;
        Look l0, l1, l2;
        look_up();
        bool h0 = found(l0);
        look_up();
        c0.load(p.cache, l0.code);
        bool h1 = found(l1);
        look_up();
        c1.load(p.cache, l1.code);
        bool h2 = found(l2);
        while (h0) {
            look_up();
            store(c0, l0);
            if (!alive) break;
            c0.load(p.cache, l2.code);
            l0 = l1;
            h0 = h1;
            l1 = l2;
            h1 = h2;
            h2 = found(l2);
            if (!h0) break;
            look_up();
            store(c1, l0);
            if (!alive) break;
            c1.load(p.cache, l2.code);
            l0 = l1;
            h0 = h1;
            l1 = l2;
            h1 = h2;
            h2 = found(l2);
        }
    } else {
        // ---------------- softmax ----------------
        const int pipe = warp >> 2;
        const int r = threadIdx.x & 127;  // row of the pipeline = lane of tensor memory
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes
        const uint32_t ts = tmem + pipe * 128 + lanes, to = tmem + kTmemO + pipe * 128 + lanes;
        int n = 0;                            // tiles of finished segments
        int items = 0, segment = 0, merges = 0, rounds = 0;
        bool alive = true;
        // The pipeline's products, issued by one thread: item t of a segment
        // that began at tile n is key tile n + t.
        const bool issuer = (threadIdx.x & 127) == 0;
        auto scores = [&](int t, bool last) {
            const int stage = (n + t) & 1;
            if (!tile_wait(p, bar(B_KFULL + stage), ((n + t) >> 1) & 1, &sh_abort)) return false;
            gemm::tmem_fence_after();
            const uint32_t qb = sbase + S::kQ + (kTwo ? pipe * S::kOperand : 0);
            const uint32_t kb = sbase + S::kK + stage * S::kOperand;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = (k >> 2) * (kTileKeys * 128) + (k & 3) * 32;
                gemm::mma_f16(tmem + pipe * 128, gemm::smem_desc(qb + off, 128),
                              gemm::smem_desc(kb + off, 128), tile_desc<kTileKeys, false>(),
                              k > 0);
            }
            gemm::mma_commit(bar(B_SFULL + pipe));
            gemm::mma_commit(bar(B_KEMPTY + stage));
            if (!kTwo && last && pipe == 0) gemm::mma_commit(bar(B_QDONE));
            return true;
        };
        auto products = [&](int t, bool started, bool last) {
            const int stage = (n + t) & 1;
            if (!tile_wait(p, bar(B_VFULL + stage), ((n + t) >> 1) & 1, &sh_abort)) return false;
            gemm::tmem_fence_after();
            const uint32_t vb = sbase + S::kV + stage * S::kOperand;
#pragma unroll
            for (int k = 0; k < kTileKeys / 16; ++k)
                mma_f16_ts(tmem + kTmemO + pipe * 128, tmem + pipe * 128 + 8 * k,
                           value_desc(vb + k * 2048), tile_desc<D, true>(), started || k > 0);
            gemm::mma_commit(bar(B_VEMPTY + stage));
            if (last) gemm::mma_commit(bar(B_ODONE + pipe));
            return true;
        };
        auto wait = [&](int b, int parity) {
            alive = tile_wait(p, bar(b), parity & 1, &sh_abort);
            alive = __all_sync(0xffffffffu, alive);
            return alive;
        };
        while (alive && walk.next()) {
            const Segment &sg = walk.sg;
            const int T = walk.t1 - walk.t0;
            const int R = sg.block * kRows + (kTwo ? pipe * kTileRows : 0) + r;
            const int tok = R / p.G, hq = sg.head * p.G + (R - tok * p.G);
            const bool live = tok < sg.s.n;
            const bool warp_live = __any_sync(0xffffffffu, live);
            if (kTwo || pipe == 0) {
                // Q in binary16, scaled by one power of two for the block: a
                // row that is not finite is left out of that and becomes NaN.
                // D / 8 lanes read a row, all of the warp's 32 at once.
                constexpr int kLanes = D / 8, kSide = 32 / kLanes, kN = 32 / kSide;
                const uint16_t *src = static_cast<const uint16_t *>(p.q.data);
                const int64_t own =
                    live ? (sg.row0 + tok) * p.q.ts + (int64_t)hq * p.q.hs : -1;
                const int chunk = lane % kLanes, side = lane / kLanes;
                uint4 w[kN];
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const int64_t at = __shfl_sync(0xffffffffu, own, i * kSide + side);
                    w[i] = make_uint4(0, 0, 0, 0);
                    if (at >= 0) w[i] = ld_past_l1(src + at + chunk * 8);
                }
                // magnitudes as the integers they sort as
                const uint32_t inf = p.bf16 ? 0x7f80u : 0x7c00u;
                uint32_t most = 0, bad = 0;  // bad: this lane's rows that are not finite, by i
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const uint32_t m2 =
                        __vmaxu2(__vmaxu2(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu),
                                 __vmaxu2(w[i].z & 0x7fff7fffu, w[i].w & 0x7fff7fffu));
                    const uint32_t m1 = max(m2 & 0xffffu, m2 >> 16);
                    const uint32_t group = (kLanes == 32 ? 0xffffffffu : (1u << (kLanes & 31)) - 1u)
                                           << (side * kLanes);
                    if (__ballot_sync(0xffffffffu, m1 >= inf) & group) bad |= 1u << i;
                    else most = max(most, m1);
                }
                most = __reduce_max_sync(0xffffffffu, most);
                if (lane == 0) {
                    const float amax = p.bf16 ? __uint_as_float(most << 16)
                                              : DT<__half>::w2f(most).x;
                    atomicMax(&sh_amax[segment & 1], __float_as_uint(amax));
                    gemm::mbar_arrive(bar(B_QMAX));
                }
                if (!wait(B_QMAX, segment)) break;
                const float by = power_of_two(13 - query_exponent(sh_amax[segment & 1]));
                if (threadIdx.x == 0) sh_amax[(segment + 1) & 1] = 0;
                const uint32_t qb = sbase + S::kQ + (kTwo ? pipe * S::kOperand : 0);
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    float x[8];
                    if (p.bf16) DT<__nv_bfloat16>::unpack(w[i], x);
                    else DT<__half>::unpack(w[i], x);
                    uint4 h = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
                    if (!((bad >> i) & 1u))
                        h = make_uint4(pack_h2(x[0] * by, x[1] * by), pack_h2(x[2] * by, x[3] * by),
                                       pack_h2(x[4] * by, x[5] * by), pack_h2(x[6] * by, x[7] * by));
                    gemm::sts128(qb + operand_at<D>((warp & 3) * 32 + i * kSide + side, chunk >> 3,
                                                    chunk & 7),
                                 h);
                }
                gemm::fence_async_shared();
                __syncwarp();
                if (lane == 0) gemm::mbar_arrive(bar(B_QREADY));
            }

            // weights are 2^(t - off), off = m - k: k lifts them so that the
            // largest weight times value scale is under 2^12 (kWeightScale),
            // and drops out of O / l
            float m = -INFINITY, l = 0.f;
            int k = 100;
            float off = -100.f;
            int done = 0;  // items of this segment
            constexpr int kEach = kTwo ? 1 : 2;
            const int t_first = kTwo ? 0 : pipe;
            if (t_first < T) {
                if (issuer)
                    alive = tile_wait(p, bar(B_QREADY), segment & 1, &sh_abort) &&
                            scores(t_first, t_first + kEach >= T);
                alive = __all_sync(0xffffffffu, alive);
                if (!alive) break;
            }
            for (int t = t_first; t < T; t += kEach) {
                if (!wait(B_SFULL + pipe, items)) break;
                if (!wait(B_INFO + ((n + t) & 3), (n + t) >> 2)) break;
                gemm::tmem_fence_after();
                const TileInfo &ti = info[(n + t) & 3];
                const int j0 = (walk.t0 + t) * kTileKeys;
                const float4 va = *reinterpret_cast<const float4 *>(ti.vmax);
                const float vm = fmaxf(fmaxf(va.x, va.y), fmaxf(va.z, va.w));
                const uint4 okw = *reinterpret_cast<const uint4 *>(ti.ok);
                uint32_t vis[4] = {okw.x, okw.y, okw.z, okw.w};
                const bool edge = (okw.x & okw.y & okw.z & okw.w) != 0xffffffffu ||
                                  j0 + kTileKeys > sg.s.ctx;  // uniform
                if (edge) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int d0 = j0 + 32 * w - sg.s.ctx;  // drafted token of bit 0
                        uint32_t see = 0;
                        if (live) see = seen_word(p, sg.row0 + tok, tok, sg.s.n, d0);
                        vis[w] &= see;
                    }
                }
                // a warp without rows leaves its weights as they are: they
                // reach no other row
                if (warp_live) {
                    // the row's largest score
                    const float top = edge ? row_top<true>(ts, ti, vis) : row_top<false>(ts, ti, vis);
                    const bool lower = vm > 0.f && vm * power_of_two(k) > kWeightScale;  // uniform
                    if (__any_sync(0xffffffffu, lower || top > m + kSlack)) {
                        if (lower) k = min(k, 11 - (int)((__float_as_uint(vm) >> 23) & 0xff) + 127);
                        const float m1 = fmaxf(m, top);
                        const float off1 = (m1 == -INFINITY ? 0.f : m1) - (float)k;
                        const float by = m == -INFINITY ? 1.f : exp2_fast(off - off1);
                        m = m1;
                        off = off1;
                        l *= by;
                        if (done) {
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) tmem_scale32(to + 32 * c, by);
                        }
                    }
                    l += edge ? row_weights<true>(ts, ti, vis, off)
                              : row_weights<false>(ts, ti, vis, off);
                }
                tmem_st_wait();
                gemm::tmem_fence_before();
                __syncwarp();
                if (lane == 0) gemm::mbar_arrive(bar(B_PFULL + pipe));
                if (issuer) {
                    alive = tile_wait(p, bar(B_PFULL + pipe), items & 1, &sh_abort) &&
                            products(t, done > 0, t + kEach >= T);
                    if (alive && t + kEach < T) alive = scores(t + kEach, t + 2 * kEach >= T);
                }
                alive = __all_sync(0xffffffffu, alive);
                if (!alive) break;
                ++items;
                ++done;
            }
            if (!alive) break;
            if (done) {
                if (!wait(B_ODONE + pipe, rounds)) break;
                ++rounds;
                gemm::tmem_fence_after();
            }
            const bool whole = walk.t0 == 0 && walk.t1 == sg.s.tiles;
            float *buf = reinterpret_cast<float *>(smem + S::kQ);  // [column][row]
            const bool joined = !kTwo && T > 1;
            if (joined && pipe == 1) {
                // this pipeline's state, over the queries once the other
                // pipeline's last scores are done as well
                if (!wait(B_QDONE, segment)) break;
                sh_ml[r] = make_float2(l, off);
                sh_m[r] = m;
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
                    const float2 o1 = sh_ml[r];
                    const float m1 = sh_m[r];
                    // both in the units of the larger offset
                    const float oo = fmaxf(m == -INFINITY ? -INFINITY : off,
                                           m1 == -INFINITY ? -INFINITY : o1.y);
                    f0 = m == -INFINITY ? 0.f : off == oo ? 1.f : exp2_fast(off - oo);
                    f1 = m1 == -INFINITY ? 0.f : o1.y == oo ? 1.f : exp2_fast(o1.y - oo);
                    l = (f0 == 0.f ? 0.f : l * f0) + (f1 == 0.f ? 0.f : o1.x * f1);
                    if (m == -INFINITY || (m1 != -INFINITY && off != oo)) {
                        m = m1;  // the offset's own maximum: their difference is k
                        off = m1 == -INFINITY ? off : o1.y;
                    }
                }
                const int64_t slot = 2 * (int64_t)blockIdx.x + (walk.t0 == 0 ? 1 : 0);
                const int64_t prow = slot * kRows + (kTwo ? pipe * kTileRows : 0) + r;
                // parts leave in units of 2^-m, without k
                const float unit = power_of_two(-k_of(off, m));
                const float by = whole ? (l == 0.f ? 0.f : 1.f / l) : unit;
                if (!whole) p.ml[prow] = make_float2(m, l * unit);
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    if (done) gemm::tmem_ld32(to + 32 * c, o);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        float v = done && f0 != 0.f ? o[j] * f0 : 0.f;
                        if (joined && f1 != 0.f) v += buf[(32 * c + j) * kTileRows + r] * f1;
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
                             whole ? -1 : part_of(cur, walk.at + sg.s.tiles - 1),
                             (int)sg.row0, sg.s.n, sg.head, sg.block, 0, 0};
            }
            gemm::tmem_fence_before();  // O is read before the next segment's products
            if (!kTwo) {
                // The pipelines begin a segment together: one that skipped
                // segments of a single tile could take an old phase of a
                // barrier for its own.
                __syncwarp();
                if (pipe == 0) {
                    if (lane == 0) gemm::mbar_arrive(bar(B_NEXT));
                } else if (!wait(B_NEXT, segment)) {
                    break;
                }
            }
            n += T;
            ++segment;
        }
        // nothing may be in flight when the tensor memory goes
        if (issuer) {
            gemm::mma_commit(bar(B_DRAIN));
            const unsigned long long t0 = gemm::now_ns();
            while (!gemm::mbar_try_wait(bar(B_DRAIN), 0))
                if (gemm::now_ns() - t0 > kWaitLimitNs) break;
        }
        __syncwarp();
    }
    gemm::tmem_fence_before();
    __syncthreads();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
}

}  // namespace tree
}  // namespace rarn
