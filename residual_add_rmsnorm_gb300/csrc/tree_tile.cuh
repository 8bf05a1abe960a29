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
//   * one thread issues tcgen05.mma: S into one of two 128-column
//     accumulators, and O += P V with P read from tensor memory and V from
//     the same row layout as K (as the transposed, N-major operand);
//   * two pipelines of four softmax warps, a thread per row: scores from
//     tensor memory, running maximum with slack, weights rounded to binary16
//     over the scores' columns.
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
constexpr int kConvWarps = 8;
constexpr int kTileThreads = 32 * (kSoftWarps + kConvWarps + 1);
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
    B_INFO = 14, B_QMAX = 18, B_QREADY = 19, B_MERGE = 20, B_DRAIN = 21, B_COUNT = 22
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

// The k of an offset m - k.
__device__ __forceinline__ int k_of(float off, float m) {
    return __float2int_rn((m == -INFINITY ? 0.f : m) - off);
}

// ---------------------------------------------------------------------------
// Converters
// ---------------------------------------------------------------------------

// A tile as a converter thread knows it: its keys' codes on the way, and what
// it needs for the values'.
template <int D>
struct Fetch {
    static constexpr int kLoads = D / 32;  // of each of K and V: 256 threads, 16 codes a load
    uint4 k[kLoads];
    int64_t code;   // where the codes of key (lane & 15) of the warp's 16 lie, < 0: nowhere
    float sc;       // lanes 0 .. 15: key scale, 16 .. 31: value scale of key (lane & 15)
    uint32_t ok;    // the warp's 16 keys that exist
    bool past;      // the tile reaches behind the context
    bool first;     // of its segment
};

// Where a converter thread's i-th load belongs: row of the tile, chunk of 16
// codes.  Eight neighbouring lanes store two rows' neighbouring chunks, which
// the swizzle keeps in different banks.
template <int D>
__device__ __forceinline__ void conv_place(int warp, int lane, int i, int &row, int &x) {
    if constexpr (D == 128) {
        row = warp * 16 + ((lane >> 2) & 3) + 4 * i;
        x = (lane & 3) | ((lane >> 4) << 2);
    } else {
        row = warp * 16 + (lane >> 2) + 8 * i;
        x = lane & 3;
    }
}

template <int D>
__device__ __forceinline__ void load_codes(const uint8_t *from, int64_t code,
                                           uint4 (&w)[Fetch<D>::kLoads]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < Fetch<D>::kLoads; ++i) {
        int row, x;
        conv_place<D>(0, lane, i, row, x);
        const int64_t at = __shfl_sync(0xffffffffu, code, row);
        w[i] = make_uint4(0, 0, 0, 0);
        if (at >= 0) w[i] = ld_stream(from + at + x * 16);
    }
}

template <int D>
__device__ __forceinline__ void fetch_tile(const Params &p, const Segment &sg, int tile, int t0,
                                           int warp, Fetch<D> &f) {
    const int lane = threadIdx.x & 31;
    const int j0 = tile * kTileKeys;
    const int j = j0 + warp * 16 + (lane & 15);
    KeyAt mine{-1, 0};
    if (j < sg.s.len) {
        const int pg = p.page_of(j);
        const int64_t page = p.table[sg.b * p.table_stride + pg];
        if (page >= 0 && page < p.cache.pages)
            mine = place(p, page, j - pg * p.cache.page_size, sg.head);
        else
            atomicOr(p.watchdog, kv::kWatchIndex);
    }
    f.ok = __ballot_sync(0xffffffffu, mine.code >= 0) & 0xffffu;
    f.past = j0 + kTileKeys > sg.s.ctx;
    f.first = tile == t0;
    f.code = mine.code;
    f.sc = 0.f;
    if (mine.code >= 0) f.sc = (lane < 16 ? p.cache.k_scale : p.cache.v_scale)[mine.scale];
    load_codes<D>(p.cache.k, mine.code, f.k);
}

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
            gemm::mbar_init(bar(B_KEMPTY + i), 1);
            gemm::mbar_init(bar(B_VFULL + i), kConvWarps);
            gemm::mbar_init(bar(B_VEMPTY + i), 1);
            gemm::mbar_init(bar(B_SFULL + i), 1);
            gemm::mbar_init(bar(B_PFULL + i), 4);
            gemm::mbar_init(bar(B_ODONE + i), 1);
        }
        for (int i = 0; i < 4; ++i) gemm::mbar_init(bar(B_INFO + i), kConvWarps);
        gemm::mbar_init(bar(B_QMAX), kTwo ? 8 : 4);
        gemm::mbar_init(bar(B_QREADY), kTwo ? 8 : 4);
        gemm::mbar_init(bar(B_MERGE), 4);
        gemm::mbar_init(bar(B_DRAIN), 1);
        gemm::fence_async_shared();
        sh_abort = 0;
        sh_nonfinite = 0;
        sh_amax[0] = sh_amax[1] = 0;
    }
    if (warp == kSoftWarps + kConvWarps) {
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

    if (warp >= kSoftWarps && warp < kSoftWarps + kConvWarps) {
        // ---------------- converters ----------------
        const int cw = warp - kSoftWarps;
        // the stream of tiles over all segments: keys two ahead, values one
        Fetch<D> f[2];
        uint4 v[Fetch<D>::kLoads];
        int tile = 0;
        bool more = walk.next();
        if (more) tile = walk.t0;
        int segments = 0;  // begun by the tiles stored
        auto fetch = [&](Fetch<D> &x) {
            if (!more) return false;
            fetch_tile<D>(p, walk.sg, tile, walk.t0, cw, x);
            if (++tile >= walk.t1) {
                more = walk.next();
                tile = walk.t0;
            }
            return true;
        };
        bool alive = true;
        int n = 0;  // tiles stored
        auto store = [&](Fetch<D> &x) {
            const int stage = n & 1;
            const uint32_t parity = ((n >> 1) & 1) ^ 1;
            TileInfo &ti = info[n & 3];
            const uint32_t kbase = sbase + S::kK + stage * S::kOperand;
            const uint32_t vbase = sbase + S::kV + stage * S::kOperand;
            alive = alive && tile_wait(p, bar(B_KEMPTY + stage), parity, &sh_abort);
            if (x.first) {
                // the scaling of this segment's queries goes into the key scales
                alive = alive && tile_wait(p, bar(B_QREADY), segments & 1, &sh_abort);
                ++segments;
            }
            alive = __all_sync(0xffffffffu, alive);
            if (!alive) return;
            const float undo =
                power_of_two(query_exponent(sh_amax[(segments - 1) & 1]) - 13) * p.scale_log2;
            const float vabs = fabsf(x.sc);
            const float vmax = warp_max(lane >= 16 && vabs < INFINITY ? vabs : 0.f);
            if (lane < 16) ti.kk[cw * 16 + lane] = x.sc * undo;
            else ti.vs[cw * 16 + lane - 16] = x.sc;
            if (lane == 0) {
                ti.vmax[cw] = vmax;
                ti.ok[cw] = (uint16_t)x.ok;
            }
#pragma unroll
            for (int i = 0; i < Fetch<D>::kLoads; ++i) {
                int row, ch;
                conv_place<D>(cw, lane, i, row, ch);
                store_codes<D, kE5M2>(kbase, row, ch, x.k[i]);
            }
            gemm::fence_async_shared();
            __syncwarp();
            if (lane == 0) gemm::mbar_arrive(bar(B_KFULL + stage));
            // Behind the context a value may be hidden from some rows, and 0
            // times NaN or infinity would reach them: such elements become
            // zero here and are added at the end to the rows that see them.
            if (x.past) {
                bool any = false;
#pragma unroll
                for (int i = 0; i < Fetch<D>::kLoads; ++i) {
                    const uint4 c = v[i];
                    v[i] = make_uint4(finite_codes<kE5M2>(c.x), finite_codes<kE5M2>(c.y),
                                      finite_codes<kE5M2>(c.z), finite_codes<kE5M2>(c.w));
                    any |= c.x != v[i].x || c.y != v[i].y || c.z != v[i].z || c.w != v[i].w;
                }
                if (any) sh_nonfinite = 1;
            }
            __syncwarp();
            if (lane == 0) gemm::mbar_arrive(bar(B_INFO + (n & 3)));
            alive = tile_wait(p, bar(B_VEMPTY + stage), parity, &sh_abort);
            alive = __all_sync(0xffffffffu, alive);
            if (!alive) return;
#pragma unroll
            for (int i = 0; i < Fetch<D>::kLoads; ++i) {
                int row, ch;
                conv_place<D>(cw, lane, i, row, ch);
                store_codes<D, kE5M2>(vbase, row, ch, v[i]);
            }
            gemm::fence_async_shared();
            __syncwarp();
            if (lane == 0) gemm::mbar_arrive(bar(B_VFULL + stage));
            ++n;
        };
        bool h0 = fetch(f[0]), h1 = fetch(f[1]);
        if (h0) load_codes<D>(p.cache.v, f[0].code, v);
        while (alive && h0) {
            store(f[0]);
            if (h1) load_codes<D>(p.cache.v, f[1].code, v);
            h0 = fetch(f[0]);
            if (!h1 || !alive) break;
            store(f[1]);
            if (h0) load_codes<D>(p.cache.v, f[0].code, v);
            h1 = fetch(f[1]);
        }
    } else if (warp == kSoftWarps + kConvWarps) {
        // ---------------- products ----------------
        if (lane == 0) {
            int n = 0;            // tiles of finished segments
            int items[2] = {0, 0};  // of each pipeline, in all
            int segment = 0;
            bool alive = true;
            while (alive && walk.next()) {
                const int T = walk.t1 - walk.t0, U = kTwo ? 2 * T : T;
                alive = tile_wait(p, bar(B_QREADY), segment & 1, &sh_abort);
                auto scores = [&](int u) {
                    const int t = kTwo ? u >> 1 : u, i = u & 1, stage = (n + t) & 1;
                    if (!kTwo || i == 0)
                        alive = alive && tile_wait(p, bar(B_KFULL + stage), ((n + t) >> 1) & 1,
                                                   &sh_abort);
                    if (!alive) return;
                    gemm::tmem_fence_after();
                    const uint32_t qb = sbase + S::kQ + (kTwo ? i * S::kOperand : 0);
                    const uint32_t kb = sbase + S::kK + stage * S::kOperand;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = (k >> 2) * (kTileKeys * 128) + (k & 3) * 32;
                        gemm::mma_f16(tmem + i * 128, gemm::smem_desc(qb + off, 128),
                                      gemm::smem_desc(kb + off, 128),
                                      tile_desc<kTileKeys, false>(), k > 0);
                    }
                    gemm::mma_commit(bar(B_SFULL + i));
                    if (!kTwo || i == 1) gemm::mma_commit(bar(B_KEMPTY + stage));
                };
                for (int u = 0; u < 2 && u < U; ++u) scores(u);
                for (int u = 0; alive && u < U; ++u) {
                    const int t = kTwo ? u >> 1 : u, i = u & 1, stage = (n + t) & 1;
                    alive = tile_wait(p, bar(B_PFULL + i), items[i] & 1, &sh_abort);
                    if (!kTwo || i == 0)
                        alive = alive && tile_wait(p, bar(B_VFULL + stage), ((n + t) >> 1) & 1,
                                                   &sh_abort);
                    if (!alive) break;
                    ++items[i];
                    gemm::tmem_fence_after();
                    const uint32_t vb = sbase + S::kV + stage * S::kOperand;
                    const bool started = kTwo ? t > 0 : u > 1;
#pragma unroll
                    for (int k = 0; k < kTileKeys / 16; ++k)
                        mma_f16_ts(tmem + kTmemO + i * 128, tmem + i * 128 + 8 * k,
                                   value_desc(vb + k * 2048), tile_desc<D, true>(),
                                   started || k > 0);
                    if (!kTwo || i == 1) gemm::mma_commit(bar(B_VEMPTY + stage));
                    if (u + 2 >= U) gemm::mma_commit(bar(B_ODONE + i));
                    if (u + 2 < U) scores(u + 2);
                }
                n += T;
                ++segment;
            }
            // nothing may be in flight when the tensor memory goes
            gemm::mma_commit(bar(B_DRAIN));
            const unsigned long long t0 = gemm::now_ns();
            while (!gemm::mbar_try_wait(bar(B_DRAIN), 0))
                if (gemm::now_ns() - t0 > kWaitLimitNs) break;
        }
        __syncwarp();
    } else {
        // ---------------- softmax ----------------
        const int pipe = warp >> 2;
        const int r = threadIdx.x & 127;  // row of the pipeline = lane of tensor memory
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes
        const uint32_t ts = tmem + pipe * 128 + lanes, to = tmem + kTmemO + pipe * 128 + lanes;
        int n = 0;                            // tiles of finished segments
        int items = 0, segment = 0, merges = 0, rounds = 0;
        bool alive = true;
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
            if (kTwo || pipe == 0) {
                // Q in binary16, scaled by one power of two for the block: a
                // row that is not finite is left out of that and becomes NaN
                const uint16_t *src = static_cast<const uint16_t *>(p.q.data) +
                                      (sg.row0 + tok) * p.q.ts + (int64_t)hq * p.q.hs;
                auto q8 = [&](int e, float (&x)[8]) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (live) w = ld_stream(src + e);
                    if (p.bf16) DT<__nv_bfloat16>::unpack(w, x);
                    else DT<__half>::unpack(w, x);
                };
                float amax = 0.f;
                bool finite = true;
#pragma unroll 4
                for (int e = 0; e < D; e += 8) {
                    float x[8];
                    q8(e, x);
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        amax = fmaxf(amax, fabsf(x[u]));
                        finite = finite && fabsf(x[u]) < INFINITY;
                    }
                }
                amax = warp_max(finite ? amax : 0.f);
                if (lane == 0) {
                    atomicMax(&sh_amax[segment & 1], __float_as_uint(amax));
                    gemm::mbar_arrive(bar(B_QMAX));
                }
                if (!wait(B_QMAX, segment)) break;
                const float by = power_of_two(13 - query_exponent(sh_amax[segment & 1]));
                if (threadIdx.x == 0) sh_amax[(segment + 1) & 1] = 0;
                const uint32_t qb = sbase + S::kQ + (kTwo ? pipe * S::kOperand : 0);
#pragma unroll 4
                for (int e = 0; e < D; e += 8) {
                    float x[8];
                    q8(e, x);
                    uint4 w = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
                    if (finite)
                        w = make_uint4(pack_h2(x[0] * by, x[1] * by), pack_h2(x[2] * by, x[3] * by),
                                       pack_h2(x[4] * by, x[5] * by), pack_h2(x[6] * by, x[7] * by));
                    gemm::sts128(qb + operand_at<D>(r, e >> 6, (e & 63) >> 3), w);
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
            for (int t = kTwo ? 0 : pipe; t < T; t += kTwo ? 1 : 2) {
                if (!wait(B_SFULL + pipe, items)) break;
                if (!wait(B_INFO + ((n + t) & 3), (n + t) >> 2)) break;
                gemm::tmem_fence_after();
                const TileInfo &ti = info[(n + t) & 3];
                const int j0 = (walk.t0 + t) * kTileKeys;
                const float4 va = *reinterpret_cast<const float4 *>(ti.vmax),
                             vb = *reinterpret_cast<const float4 *>(ti.vmax + 4);
                const float vm = fmaxf(fmaxf(fmaxf(va.x, va.y), fmaxf(va.z, va.w)),
                                       fmaxf(fmaxf(vb.x, vb.y), fmaxf(vb.z, vb.w)));
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
                // the row's largest score
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float s[32];
                    gemm::tmem_ld32(ts + 32 * c, s);
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 kk = *reinterpret_cast<const float4 *>(ti.kk + 32 * c + j);
                        float a0 = s[j] * kk.x, a1 = s[j + 1] * kk.y, a2 = s[j + 2] * kk.z,
                              a3 = s[j + 3] * kk.w;
                        if (edge) {
                            if (!((vis[c] >> j) & 1u)) a0 = -INFINITY;
                            if (!((vis[c] >> (j + 1)) & 1u)) a1 = -INFINITY;
                            if (!((vis[c] >> (j + 2)) & 1u)) a2 = -INFINITY;
                            if (!((vis[c] >> (j + 3)) & 1u)) a3 = -INFINITY;
                        }
                        top = fmaxf(top, fmaxf(fmaxf(a0, a1), fmaxf(a2, a3)));
                    }
                }
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
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float s[32];
                    gemm::tmem_ld32(ts + 32 * c, s);
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 kk = *reinterpret_cast<const float4 *>(ti.kk + 32 * c + j);
                        const float4 vs = *reinterpret_cast<const float4 *>(ti.vs + 32 * c + j);
                        float q0 = fmaf(s[j], kk.x, -off), q1 = fmaf(s[j + 1], kk.y, -off),
                              q2 = fmaf(s[j + 2], kk.z, -off), q3 = fmaf(s[j + 3], kk.w, -off);
                        const uint32_t v4 = edge ? vis[c] >> j : 0xfu;
                        if (edge) {
                            if (!(v4 & 1u)) q0 = -INFINITY;
                            if (!(v4 & 2u)) q1 = -INFINITY;
                            if (!(v4 & 4u)) q2 = -INFINITY;
                            if (!(v4 & 8u)) q3 = -INFINITY;
                        }
                        q0 = exp2_fast(q0);
                        q1 = exp2_fast(q1);
                        q2 = exp2_fast(q2);
                        q3 = exp2_fast(q3);
                        l += (q0 + q1) + (q2 + q3);
                        q0 *= vs.x;
                        q1 *= vs.y;
                        q2 *= vs.z;
                        q3 *= vs.w;
                        if (edge) {
                            if (!(v4 & 1u)) q0 = 0.f;
                            if (!(v4 & 2u)) q1 = 0.f;
                            if (!(v4 & 4u)) q2 = 0.f;
                            if (!(v4 & 8u)) q3 = 0.f;
                        }
                        w[j / 2] = pack_h2(q0, q1);
                        w[j / 2 + 1] = pack_h2(q2, q3);
                    }
                    tmem_st16(ts + 16 * c, w);
                }
                tmem_st_wait();
                gemm::tmem_fence_before();
                __syncwarp();
                if (lane == 0) gemm::mbar_arrive(bar(B_PFULL + pipe));
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
                // this pipeline's state, over the queries (every product of
                // the segment is done)
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
            n += T;
            ++segment;
        }
    }
    gemm::tmem_fence_before();
    __syncthreads();
    if (warp == kSoftWarps + kConvWarps)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
}

}  // namespace tree
}  // namespace rarn
