// kv_rows.cuh -- per-head RMSNorm of queries and keys with the position
// rotation, and the 8-bit cache's write and read.
//
//   n = x * rsqrt(mean(x^2) + eps) * gamma       over one head's D elements
//   (a, b) -> (a cos - b sin, b cos + a sin)     for the first `rot` elements,
//                                                pairs (i, i + rot / 2) or (2i, 2i + 1)
//   code = RN(n / s)                             s given
//   code = RN((n * (1 / max|n|)) * maxf)         per row, s = max|n| / maxf
//
// All of it is one pass: a head is 128 to 512 bytes, so the row's elements
// stay in registers between the sum of squares, the rotation and the row's
// largest magnitude, and memory is touched once per byte.
//
// Vector kernel.  A lane owns two 16-byte packs that hold both halves of its
// rotation pairs (pack p and pack rot / 2 + p for "half" pairs, two
// neighbouring packs otherwise), so the rotation needs no exchange; a group
// of D / (2 packs) lanes, rounded up to a power of two, owns a head and
// reduces by shuffles inside itself.  A warp walks over heads of one tensor
// and token, loading the next two heads of each group while it works on two:
// the products of gamma with the token's cosines and sines, which every head
// shares, stay in registers, and a head costs six multiply-adds per pair
// (packed two to an instruction they measured no faster; the table is
// binary32: read per head its 8 D bytes would be four times the head's own).
//
// Bound by memory: 8192 tokens of 64 + 8 heads of 128, bfloat16, take 57.6 us
// (5.3 TB/s, 78 % of a copy's rate) and 64.5 us with the keys and values
// written to the cache (74 %); what is missing is where a warp ends and the
// next has its first loads under way.  One token takes 4.9 us, a launch and two
// dependent loads.
#pragma once

#include "kv.cuh"

namespace rarn {
namespace kv {

struct RowParams {
    Heads q, k, v;          // inputs; heads == 0: none
    Heads q_out, k_out;     // k_out.data == nullptr: keys go to the cache only
    const void *q_gamma, *k_gamma;  // [D] or nullptr: no norm
    const float *table;     // [table_rows, rot]: cos then sin; nullptr: no rotation
    const int64_t *positions;
    int64_t table_rows;
    int rot;
    int interleaved;
    const int64_t *slots;   // cache slot of each token, < 0: not written
    Cache cache;            // cache.k == nullptr: none
    int64_t T;
    int D;
    float eps;
    unsigned int *watchdog;
};

// What becomes of one tensor's heads of a token.
struct Role {
    const char *src;        // the token's first head
    char *dst;              // 16- or 32-bit output, or nullptr
    const void *gamma;
    int64_t src_hs, dst_hs; // elements between heads
    uint8_t *codes;         // the cache's codes at head 0 of slot 0 of page 0, or nullptr
    float *scales;
    int heads;
    bool rotate;
};

enum Tensor : int { T_Q = 0, T_K = 1, T_V = 2 };

template <typename T>
__device__ __forceinline__ Role role_of(const RowParams &p, int64_t t, int which) {
    Role r{};
    const Heads &in = which == T_Q ? p.q : which == T_K ? p.k : p.v;
    r.src = static_cast<const char *>(in.data) + t * in.ts * (int64_t)sizeof(T);
    r.src_hs = in.hs;
    r.heads = in.heads;
    if (which != T_V) {
        const Heads &out = which == T_Q ? p.q_out : p.k_out;
        if (out.data) r.dst = static_cast<char *>(out.data) + t * out.ts * (int64_t)sizeof(T);
        r.dst_hs = out.hs;
        r.gamma = which == T_Q ? p.q_gamma : p.k_gamma;
        r.rotate = p.table != nullptr;
    }
    if (which != T_Q && p.cache.k) {
        r.codes = which == T_K ? p.cache.k : p.cache.v;
        r.scales = which == T_K ? p.cache.k_scale : p.cache.v_scale;
    }
    return r;
}

// A token's place in the cache: page and slot inside it; page < 0: none.
struct Place {
    int64_t page;
    int at;
};

__device__ __forceinline__ Place place_of(const RowParams &p, int64_t slot, bool reporter) {
    Place pl{-1, 0};
    if (slot < 0) return pl;
    const int64_t page = slot / p.cache.page_size;
    if (page >= p.cache.pages) {
        if (reporter) atomicOr(p.watchdog, kWatchIndex);
        return pl;
    }
    pl.page = page;
    pl.at = static_cast<int>(slot - page * p.cache.page_size);
    return pl;
}

// The row of the rotation table for a position; nullptr with *ok = false when its
// position lies outside the table (the token's rows are then left as they are).
__device__ __forceinline__ const float *table_row(const RowParams &p, int64_t pos, bool reporter,
                                                  bool *ok) {
    *ok = true;
    if (!p.table) return nullptr;
    if (pos < 0 || pos >= p.table_rows) {
        if (reporter) atomicOr(p.watchdog, kWatchIndex);
        *ok = false;
        return nullptr;
    }
    return p.table + pos * p.rot;
}

template <int LG>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int m = LG / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

template <int LG>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int m = LG / 2; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, m));
    return v;
}

// A row's multipliers and scale from its largest magnitude: the 8-bit output
// forms' rule (quant_row).
__device__ __forceinline__ QMul row_mul(float amax, int fmt, float *scale) {
    const float maxf = q_maxf(fmt);
    *scale = amax > 0.f ? amax / maxf : 1.f;
    if (!(amax > 0.f)) return QMul{1.f, 1.f};
    const float k = amax < 1.17549435e-38f ? 16777216.f : 1.f;
    return QMul{1.f / (amax * k), maxf * k};
}

// A lane's 2 E elements as the first and second members of its E pairs: half
// style, pack a against pack b; interleaved, even elements against odd ones.
template <typename T, bool kInter>
struct Pairs {
    static constexpr int E = DT<T>::EPV;
    float a[E], b[E];

    __device__ __forceinline__ void unpack(const uint4 &pa, const uint4 &pb) {
        float x[E], y[E];
        DT<T>::unpack(pa, x);
        DT<T>::unpack(pb, y);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            if constexpr (kInter) {
                const float *z = 2 * j < E ? x + 2 * j : y + (2 * j - E);
                a[j] = z[0];
                b[j] = z[1];
            } else {
                a[j] = x[j];
                b[j] = y[j];
            }
        }
    }

    // The elements in memory order.
    __device__ __forceinline__ void elements(float (&x)[E], float (&y)[E]) const {
#pragma unroll
        for (int j = 0; j < E; ++j) {
            if constexpr (kInter) {
                float *z = 2 * j < E ? x + 2 * j : y + (2 * j - E);
                z[0] = a[j];
                z[1] = b[j];
            } else {
                x[j] = a[j];
                y[j] = b[j];
            }
        }
    }
};

// Heads of a group that are loaded at a time, ahead of as many being worked
// on, and CTAs per SM (at most 102 registers a thread).  Measured, bfloat16,
// 8192 tokens of 64 + 8 heads of 128: 57.9 us; one head at a time 63.6 (60.3
// with six CTAs), four CTAs 61.2.
constexpr int kAtATime = 2;
constexpr int kRowCtas = 5;

// A warp: one token, `per` heads of one tensor for each group of LG lanes.
// The work items of a token are its tensors' chunks of per * 32 / LG heads,
// `chunks` in all (nq of q, then nk of k, then those of v).
template <typename T, int LG, bool kInter>
__global__ void __launch_bounds__(128, kRowCtas)
    k_head_rows(const RowParams p, int per, int nq, int nk, int chunks) {
    constexpr int E = DT<T>::EPV;  // elements per pack
    constexpr int GPW = 32 / LG;   // groups per warp
    grid_dependency_wait();
    grid_launch_dependents();
    // a CTA's warps take the same chunk of four tokens, so they end together
    const unsigned block = blockIdx.x / (unsigned)chunks;
    const int64_t t = (int64_t)block * 4 + (threadIdx.x >> 5);
    if (t >= p.T) return;  // whole warps
    const int lane = threadIdx.x & 31, l = lane % LG;
    int chunk = static_cast<int>(blockIdx.x - block * chunks);
    const int which = chunk < nq ? T_Q : chunk < nq + nk ? T_K : T_V;
    chunk -= which == T_Q ? 0 : which == T_K ? nq : nq + nk;
    const Role r = role_of<T>(p, t, which);
    const int h0 = chunk * (per * GPW) + lane / LG;
    const int end = min(r.heads, (chunk + 1) * (per * GPW));

    // this lane's two packs
    const bool owns = l < p.D / (2 * E);
    const bool turns = r.rotate && l < p.rot / (2 * E);
    // past the rotated lanes neighbouring packs in either style
    const int ea = turns && !kInter ? l * E : 2 * E * l;
    const int eb = turns && !kInter ? p.rot / 2 + l * E : ea + E;

    // first what the other loads wait for
    const int64_t pos = p.table ? p.positions[t] : 0;
    const int64_t slot = r.codes ? p.slots[t] : -1;
    const T *src = reinterpret_cast<const T *>(r.src);
    auto load = [&](int h, uint4 &a, uint4 &b) {
        a = b = make_uint4(0, 0, 0, 0);
        if (owns && h < end) {
            const T *s = src + h * r.src_hs;
            a = ld_stream(s + ea);
            b = ld_stream(s + eb);
        }
    };
    constexpr int U = kAtATime;
    uint4 xa[U], xb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) load(h0 + u * GPW, xa[u], xb[u]);

    bool ok;
    const float *tr = table_row(p, pos, lane == 0, &ok);
    if (!ok) return;  // the whole warp: one token
    const Place pl = place_of(p, slot, lane == 0);
    // gamma, and its products with the cosines and sines
    Pairs<T, kInter> g;
    float bs[E], as[E];  // -gamma_b sin, gamma_a sin; times cos they stay in g
    {
#pragma unroll
        for (int j = 0; j < E; ++j) g.a[j] = g.b[j] = 1.f;
        if (r.gamma && owns)
            g.unpack(ld_keep(static_cast<const T *>(r.gamma) + ea),
                     ld_keep(static_cast<const T *>(r.gamma) + eb));
        if (turns) {
#pragma unroll
            for (int j = 0; j < E; j += 4) {
                const float4 c = __ldg(reinterpret_cast<const float4 *>(tr + l * E + j));
                const float4 s =
                    __ldg(reinterpret_cast<const float4 *>(tr + p.rot / 2 + l * E + j));
                const float cj[4] = {c.x, c.y, c.z, c.w}, sj[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    bs[j + u] = -g.b[j + u] * sj[u];
                    as[j + u] = g.a[j + u] * sj[u];
                    g.a[j + u] *= cj[u];
                    g.b[j + u] *= cj[u];
                }
            }
        }
    }
    const float inv_d = 1.f / static_cast<float>(p.D);
    const float given = r.codes && p.cache.mode == Q_TENSOR ? __ldg(r.scales) : 1.f;
    uint8_t *codes = nullptr;
    float *scales = nullptr;
    if (pl.page >= 0) {
        codes = r.codes + pl.page * p.cache.page_stride + pl.at * p.cache.slot_stride;
        scales = r.scales + pl.page * p.cache.s_page + pl.at * p.cache.s_slot;
    }

    auto head = [&](int h, const uint4 &pa, const uint4 &pb) {
        const bool live = owns && h < end;
        Pairs<T, kInter> x;
        x.unpack(pa, pb);
        float inv = 1.f;
        if (r.gamma) {  // uniform
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < E; ++j) ss = fmaf(x.b[j], x.b[j], fmaf(x.a[j], x.a[j], ss));
            inv = rsqrtf(fmaf(group_sum<LG>(ss), inv_d, p.eps));
        }
        if (turns) {
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float a = fmaf(x.b[j], bs[j], x.a[j] * g.a[j]);
                const float b = fmaf(x.a[j], as[j], x.b[j] * g.b[j]);
                x.a[j] = a * inv;
                x.b[j] = b * inv;
            }
        } else if (r.gamma) {
#pragma unroll
            for (int j = 0; j < E; ++j) {
                x.a[j] = x.a[j] * inv * g.a[j];
                x.b[j] = x.b[j] * inv * g.b[j];
            }
        }
        float fa[E], fb[E];
        x.elements(fa, fb);
        if (live && r.dst) {
            T *d = reinterpret_cast<T *>(r.dst) + h * r.dst_hs;
            st_global(d + ea, DT<T>::pack(fa));
            st_global(d + eb, DT<T>::pack(fb));
        }
        if (codes) {  // uniform
            if (p.cache.mode == Q_ROW) {
                float amax = 0.f;
#pragma unroll
                for (int j = 0; j < E; ++j) amax = fmaxf(amax, fmaxf(fabsf(fa[j]), fabsf(fb[j])));
                amax = group_max<LG>(amax);
                float scale;
                const QMul m = row_mul(amax, p.cache.fmt, &scale);
                if (l == 0 && live) scales[h * p.cache.s_head] = scale;
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    fa[j] = (fa[j] * m.m1) * m.m2;
                    fb[j] = (fb[j] * m.m1) * m.m2;
                }
            } else {
                // divided: a reciprocal's rounding would move ties, and that of
                // a subnormal scale is infinite
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    fa[j] /= given;
                    fb[j] /= given;
                }
            }
            if (live) {
                uint8_t *d = codes + h * p.cache.head_stride;
                st_codes<E>(d + ea, fa, p.cache.fmt);
                st_codes<E>(d + eb, fb, p.cache.fmt);
            }
        }
    };
    // groups whose heads have run out go along with the warp's reductions
    const int first = chunk * (per * GPW);
#pragma unroll 1
    for (int i = 0; first + i < end; i += U * GPW) {
        uint4 na[U], nb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) load(h0 + i + (U + u) * GPW, na[u], nb[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (first + i + u * GPW < end) head(h0 + i + u * GPW, xa[u], xb[u]);  // uniform
            xa[u] = na[u];
            xb[u] = nb[u];
        }
    }
}

// Any head size, rotation width, stride and alignment: a warp per head, a
// lane per rotation pair (then per unrotated element), the row re-read from
// L1 for each of its passes.
template <typename T>
__global__ void __launch_bounds__(128) k_head_rows_any(const RowParams p, int heads) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t t = item / heads;
    if (t >= p.T) return;
    const int lane = threadIdx.x & 31;
    int h = static_cast<int>(item - t * heads);
    int which = T_Q;
    if (h >= p.q.heads) {
        h -= p.q.heads;
        which = T_K;
        if (h >= p.k.heads) {
            h -= p.k.heads;
            which = T_V;
        }
    }
    const Role r = role_of<T>(p, t, which);
    bool ok;
    const float *tr = table_row(p, p.table ? p.positions[t] : 0, lane == 0, &ok);
    if (!ok) return;
    const Place pl = place_of(p, r.codes ? p.slots[t] : -1, lane == 0);
    const T *src = reinterpret_cast<const T *>(r.src) + h * r.src_hs;
    float inv = 1.f;
    if (r.gamma) {
        float ss = 0.f;
        for (int e = lane; e < p.D; e += 32) {
            const float x = DT<T>::to_f(src[e]);
            ss = fmaf(x, x, ss);
        }
        inv = rsqrtf(fmaf(warp_sum(ss), 1.f / static_cast<float>(p.D), p.eps));
    }
    const bool turn = r.rotate && tr;
    const int half = turn ? p.rot / 2 : 0;
    const int work = half + (p.D - 2 * half);  // pairs, then single elements
    auto normed = [&](int e) {
        const float x = DT<T>::to_f(src[e]);
        return r.gamma ? x * inv * ld_elem<T>(r.gamma, e) : x;
    };
    // element(s) of work item i: one rotated pair or one element
    auto value = [&](int i, int &e0, int &e1, float &a, float &b) {
        if (i < half) {
            e0 = p.interleaved ? 2 * i : i;
            e1 = p.interleaved ? 2 * i + 1 : half + i;
            const float x = normed(e0), y = normed(e1);
            const float c = __ldg(tr + i), s = __ldg(tr + half + i);
            a = x * c - y * s;
            b = y * c + x * s;
        } else {
            e0 = half + i;
            e1 = -1;
            a = normed(e0);
            b = 0.f;
        }
    };
    QMul m{1.f, 1.f};
    float given = 1.f;
    const bool store_codes = pl.page >= 0;
    if (store_codes) {
        if (p.cache.mode == Q_ROW) {
            float amax = 0.f;
            for (int i = lane; i < work; i += 32) {
                int e0, e1;
                float a, b;
                value(i, e0, e1, a, b);
                amax = fmaxf(amax, fmaxf(fabsf(a), fabsf(b)));
            }
            amax = warp_max(amax);
            float scale;
            m = row_mul(amax, p.cache.fmt, &scale);
            if (lane == 0)
                r.scales[pl.page * p.cache.s_page + h * p.cache.s_head +
                         pl.at * p.cache.s_slot] = scale;
        } else {
            given = __ldg(r.scales);
        }
    }
    uint8_t *codes = store_codes ? r.codes + pl.page * p.cache.page_stride +
                                       h * p.cache.head_stride + pl.at * p.cache.slot_stride
                                 : nullptr;
    for (int i = lane; i < work; i += 32) {
        int e0, e1;
        float a, b;
        value(i, e0, e1, a, b);
        if (r.dst) {
            T *d = reinterpret_cast<T *>(r.dst) + h * r.dst_hs;
            d[e0] = DT<T>::from_f(a);
            if (e1 >= 0) d[e1] = DT<T>::from_f(b);
        }
        if (codes) {
            if (p.cache.mode == Q_ROW) {
                a = (a * m.m1) * m.m2;
                b = (b * m.m1) * m.m2;
            } else {
                a /= given;
                b /= given;
            }
            codes[e0] = fp8x1(a, p.cache.fmt);
            if (e1 >= 0) codes[e1] = fp8x1(b, p.cache.fmt);
        }
    }
}

// ---------------------------------------------------------------------------
// The cache read back: x = RN(code * s), sequences packed one after another.
// ---------------------------------------------------------------------------
struct ReadParams {
    Heads k_out, v_out;      // [rows, heads, D]
    Cache cache;
    const int32_t *table;    // [B, width] pages of each sequence
    int64_t table_stride;
    int table_width;
    const int32_t *starts;   // [B + 1]: first output row of each sequence
    int B;
    int64_t rows;
    int D;
    unsigned int *watchdog;
};

constexpr int kReadThreads = 256;

// A whole 32-byte sector: two 16-byte stores of it from one lane, half a sector
// each, cost L2 a merge.
__device__ __forceinline__ void st_global32(void *p, const uint4 &a, const uint4 &b) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y),
                 "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

// Each CTA finds the cache place of its kReadRows rows once (a binary search
// over the sequences' starts), then streams their codes, 16 to a load, and
// stores 32 bytes of 16-bit values at a time.  Bound by memory: 32 sequences
// of up to 4096 tokens, 8 heads of 128, row scales, 68 us for 409 MB (89 % of
// a copy's rate); with two 16-byte stores a piece 78.6 us, with the piece's
// indices divided out anew for every load 83.9.
// kStore: bytes of a store, 0 for element by element.
template <typename T, int kStore, bool kE5M2, int kReadRows>
__global__ void __launch_bounds__(kReadThreads) k_cache_read(const ReadParams p) {
    __shared__ int64_t s_code[kReadRows], s_scale[kReadRows];  // offsets; code < 0: nothing
    __shared__ int s_state[kReadRows];                         // 0: leave, 1: read, 2: zeros
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t r0 = (int64_t)blockIdx.x * kReadRows;
    if (threadIdx.x < kReadRows) {
        const int64_t r = r0 + threadIdx.x;
        int state = 0;
        int64_t code = 0, scale = 0;
        // the last sequence that starts at or before row r
        int lo = 0, hi = p.B;  // starts[lo] <= r < starts[hi]
        if (r < p.rows && r >= p.starts[0] && r < p.starts[p.B]) {
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (p.starts[mid] <= r) lo = mid;
                else hi = mid;
            }
            const int64_t j = r - p.starts[lo];
            const int64_t pg = j / p.cache.page_size;
            const int at = static_cast<int>(j - pg * p.cache.page_size);
            state = 2;
            if (pg < p.table_width) {
                const int64_t page = p.table[lo * p.table_stride + pg];
                if (page >= 0 && page < p.cache.pages) {
                    state = 1;
                    code = page * p.cache.page_stride + at * p.cache.slot_stride;
                    scale = page * p.cache.s_page + at * p.cache.s_slot;
                }
            }
            if (state == 2) atomicOr(p.watchdog, kWatchIndex);
        }
        s_code[threadIdx.x] = code;
        s_scale[threadIdx.x] = scale;
        s_state[threadIdx.x] = state;
    }
    __syncthreads();
    // A thread keeps to one 16-code piece of the rows (key or value, head, place
    // in the head), so that only the row's offsets change from load to load.
    const int per_head = p.D / 16;
    const int per_row = 2 * p.cache.heads * per_head;
    const int side = per_row < kReadThreads ? kReadThreads / per_row : 1;  // rows side by side
    const int mine = threadIdx.x % per_row;
    const int first = threadIdx.x / per_row;
    if (first >= side) return;
    constexpr int U = 4;
    for (int x = per_row < kReadThreads ? mine : threadIdx.x; x < per_row; x += kReadThreads) {
        const int hh = x / per_head, piece = x - hh * per_head;
        const bool val = hh >= p.cache.heads;
        const int h = val ? hh - p.cache.heads : hh;
        const uint8_t *codes =
            (val ? p.cache.v : p.cache.k) + h * p.cache.head_stride + piece * 16;
        const float *scales = (val ? p.cache.v_scale : p.cache.k_scale) + h * p.cache.s_head;
        const Heads &o = val ? p.v_out : p.k_out;
        T *out = static_cast<T *>(o.data) + r0 * o.ts + h * o.hs + piece * 16;
        const int start = per_row < kReadThreads ? first : 0;
        for (int row0 = start; row0 < kReadRows; row0 += U * side) {
            uint4 w[U];
            float sc[U];
            int state[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int row = row0 + u * side;
                state[u] = row < kReadRows ? s_state[row] : 0;
                w[u] = make_uint4(0, 0, 0, 0);
                sc[u] = 0.f;
                if (state[u] == 1) {
                    w[u] = ld_stream(codes + s_code[row]);
                    sc[u] = scales[s_scale[row]];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (state[u] == 0) continue;
                T *d = out + (row0 + u * side) * o.ts;
                float f[16];
                const uint32_t ws[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t lo, hi;
                    codes4_to_h2<kE5M2>(ws[j], lo, hi);
                    const float2 a = DT<__half>::w2f(lo), b = DT<__half>::w2f(hi);
                    f[4 * j] = a.x * sc[u];
                    f[4 * j + 1] = a.y * sc[u];
                    f[4 * j + 2] = b.x * sc[u];
                    f[4 * j + 3] = b.y * sc[u];
                }
                if constexpr (kStore) {
                    constexpr int E = DT<T>::EPV;
                    uint4 out16[16 / E];
#pragma unroll
                    for (int j = 0; j < 16 / E; ++j) {
                        float g[E];
#pragma unroll
                        for (int e = 0; e < E; ++e) g[e] = f[j * E + e];
                        out16[j] = DT<T>::pack(g);
                    }
#pragma unroll
                    for (int j = 0; j < 16 / E; j += kStore / 16) {
                        if constexpr (kStore == 32) st_global32(d + j * E, out16[j], out16[j + 1]);
                        else st_global(d + j * E, out16[j]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) d[e] = DT<T>::from_f(f[e]);
                }
            }
        }
    }
}

// Host launchers (instantiated per storage type).
template <typename T>
cudaError_t launch_head_rows(const RowParams &p, bool vec, int num_sms, bool pdl,
                             cudaStream_t st);
template <typename T>
cudaError_t launch_cache_read(const ReadParams &p, int store, int num_sms, bool pdl,
                              cudaStream_t st);

}  // namespace kv
}  // namespace rarn
