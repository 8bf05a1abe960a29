// verify.cuh -- verification of drafted tokens against the target's probabilities
// from given random numbers, and the draw of the token behind the accepted ones.
//
// Row 0 of a sequence is its last known token, the others are drafts below a parent
// row (a chain: the row before).  With p the target's probabilities at a row and u
// its random number, a draft c below it with token x is accepted where
//   u q(x) < p(x)                        q: what the draft was drawn from (chains);
//   s <= u < s + p(x)                    without q: s sums p over the earlier siblings'
//                                        other tokens.
// From the last accepted row the next token is drawn by a second number v: the
// smallest x with w(0) + .. + w(x) > v * (w's sum), w the probabilities left there:
//   w = max(p - q, 0), or p without the refused children's tokens, or p where
//   nothing was refused or nothing is left.
// That is the target's own distribution, whatever was drafted.
//
// The draw must not hang on the order of a sum, nor on binary32's errors in a sum of
// 10^5 terms (they pass the weight of a rare token), so weights are summed as
// integers: F(w) = round(w 2^23) 2^23 + round(rest 2^46), in units of 2^-46, two
// binary32 additions of a constant whose result's bits are the integer.  Any
// split of the row gives the same sums.
//
// One row of p (and q) a sequence is all that has to be read in full, so the bound
// is memory, or for few sequences the chain of launch, indices, the accepted row, its
// sums and the draw: a cluster of CTAs takes a sequence, each a part of the row.
// Measured: 64 chains of up to 6 rows with draft probabilities, 128256 tokens, binary32,
// 13.7 us (9.7 at a copy's rate), 128 of them 22.3 us (19.3); one chain over 32000 tokens
// 5.6 us; 16 trees of up to 32 rows over 50257 tokens 7.5 us.
#pragma once

#include "kv.cuh"

namespace rarn {
namespace verify {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroup = 1024;          // neighbouring elements summed by a warp
constexpr int kMaxVocab = 1 << 20;
constexpr int kMaxGroups = kMaxVocab / kGroup;
constexpr int kMaxTree = 1024;        // rows of a sequence's tree
constexpr int kMaxCluster = 8;
constexpr int kFrac = 46;             // F's unit is 2^-kFrac

struct Params {
    const void *p, *q;          // [rows, V]; q may be nullptr
    int64_t ldp, ldq;
    const int64_t *tokens;      // [rows]
    const int32_t *parents;     // [rows] or nullptr: a chain
    const int32_t *starts;      // [B + 1]
    const float *u, *v;         // [rows], [B]
    int64_t *out_tokens;        // [B, W]
    int32_t *path, *lengths;    // [B, W], [B]
    int64_t rows;
    int B, V, W;
    bool vec;                   // rows of p and q begin on 16-byte boundaries
    unsigned int *watchdog;
};

// What is left to draw from.
enum Weights : int { W_ALL = 0, W_REST = 1, W_WITHOUT = 2 };

// 0 .. 1, NaN as 0.
__device__ __forceinline__ float unit(float x) { return __saturatef(x); }

// The two halves of F(x) as bits above those of two constants, two elements at a time,
// 0 <= x <= 1: x + 1 has x's first half in its bits above those of 1; the rest,
// exact and at most 2^-24, comes out of a sum with 1.5 * 2^-23 alike.
constexpr uint32_t kOne = 0x3f800000u;      // bits of 1
constexpr uint32_t kSmall = 0x34400000u;    // bits of 1.5 * 2^-23

__device__ __forceinline__ void halves(float2 x, float2 &hi, float2 &lo) {
    const float s = __uint_as_float(kSmall);
    hi = __fadd2_rn(x, float2{1.f, 1.f});
    const float2 first = __fadd2_rn(hi, float2{-1.f, -1.f});
    lo = __fadd2_rn(__fadd2_rn(x, float2{-first.x, -first.y}), float2{s, s});
}

__device__ __forceinline__ int64_t fixed(float x) {
    float2 hi, lo;
    halves(float2{unit(x), 0.f}, hi, lo);
    return ((int64_t)(int32_t)(__float_as_uint(hi.x) - kOne) << 23) +
           (int32_t)(__float_as_uint(lo.x) - kSmall);
}

// max(p - q, 0): F(p) - F(min(p, q)), F being monotone.
__device__ __forceinline__ int64_t weight(float p, float q, bool rest) {
    return rest ? fixed(p) - fixed(fminf(unit(p), unit(q))) : fixed(p);
}

// A lane's sum of up to 32 weights.
struct Lane {
    uint32_t hi = 0, lo = 0;

    template <bool kRest>
    __device__ __forceinline__ void add(float2 p, float2 q) {
        float2 h, l;
        p = float2{unit(p.x), unit(p.y)};
        halves(p, h, l);
        if constexpr (kRest) {
            float2 h2, l2;
            halves(float2{fminf(p.x, unit(q.x)), fminf(p.y, unit(q.y))}, h2, l2);
            hi += __float_as_uint(h.x) - __float_as_uint(h2.x);
            hi += __float_as_uint(h.y) - __float_as_uint(h2.y);
            lo += __float_as_uint(l.x) - __float_as_uint(l2.x);
            lo += __float_as_uint(l.y) - __float_as_uint(l2.y);
        } else {
            hi += __float_as_uint(h.x) - kOne;
            hi += __float_as_uint(h.y) - kOne;
            lo += __float_as_uint(l.x) - kSmall;
            lo += __float_as_uint(l.y) - kSmall;
        }
    }
    __device__ __forceinline__ int64_t sum() const {
        return ((int64_t)(int32_t)hi << 23) + (int32_t)lo;
    }
};

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// Exclusive sum over the CTA; the total to every thread.
__device__ __forceinline__ int64_t block_scan64(int64_t v, int64_t *red, int64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t in = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, in, m);
        if (lane >= m) in += a;
    }
    __syncthreads();  // red may be another call's
    if (lane == 31) red[warp] = in;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) before = all;
        all += red[w];
    }
    *total = all;
    return before + in - v;
}

// The sum of a group's weights, in every lane.  Loads come in batches of 32 registers
// (64 bytes of p and of q a lane), which four CTAs to an SM have room for.
template <typename T, bool kRest>
__device__ __forceinline__ int64_t group_sum64(const T *p, const T *q, int g, int V, bool vec) {
    constexpr int E = DT<T>::EPV;
    const int lane = threadIdx.x & 31, at = g * kGroup;
    Lane s;
    if (vec && at + kGroup <= V) {
        constexpr int N = 4;
#pragma unroll
        for (int i0 = 0; i0 < kGroup / (32 * E); i0 += N) {
            uint4 a[N], b[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                a[i] = ld_stream(p + at + ((i0 + i) * 32 + lane) * E);
                if constexpr (kRest) b[i] = ld_stream(q + at + ((i0 + i) * 32 + lane) * E);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float x[E], y[E];
                DT<T>::unpack(a[i], x);
                if constexpr (kRest) DT<T>::unpack(b[i], y);
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    s.add<kRest>(float2{x[e], x[e + 1]},
                                 kRest ? float2{y[e], y[e + 1]} : float2{0.f, 0.f});
            }
        }
    } else {
        constexpr int N = 16;
#pragma unroll 1
        for (int i0 = at + lane; i0 < min(at + kGroup, V); i0 += N * 32) {
            T a[N], b[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int x = i0 + i * 32;
                a[i] = b[i] = DT<T>::from_f(0.f);
                if (x < V) {
                    a[i] = p[x];
                    if constexpr (kRest) b[i] = q[x];
                }
            }
#pragma unroll
            for (int i = 0; i < N; i += 2)
                s.add<kRest>(float2{DT<T>::to_f(a[i]), DT<T>::to_f(a[i + 1])},
                             float2{DT<T>::to_f(b[i]), DT<T>::to_f(b[i + 1])});
        }
    }
    return warp_sum64(s.sum());
}

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// v to the same shared-memory place in CTA `rank` of the cluster.
__device__ __forceinline__ void store_peer(int64_t *place, int rank, int64_t v) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(place));
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(r), "l"(v) : "memory");
}

// A cluster of CTAs per sequence; every CTA finds the accepted rows by itself, then
// sums its part of the last one's weights.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) k_verify(const Params p, int cluster) {
    __shared__ int64_t s_group[kMaxGroups];      // weights of this CTA's groups
    __shared__ int64_t s_mass[kMaxTree];         // F(p) of each draft; 0: its token came before
    __shared__ int s_parent[kMaxTree], s_next[kMaxTree];
    __shared__ int s_token[kMaxTree], s_walk[kMaxTree];
    __shared__ int64_t red[kWarps], s_part[2][kMaxCluster];
    __shared__ int64_t s_u[kMaxTree];
    __shared__ int s_stop, s_length, s_deep, s_found, s_gone;
    grid_dependency_wait();
    grid_launch_dependents();
    cluster_arrive();  // waited for before a peer's shared memory is written
    const int b = blockIdx.x / cluster, rank = blockIdx.x - b * cluster;
    const int tid = threadIdx.x, W = p.W;
    const bool first = rank == 0;
    const int64_t lo = p.starts[b], hi = p.starts[b + 1];
    const bool tree = p.parents != nullptr;
    int64_t *tokens = p.out_tokens + (int64_t)b * W;
    int32_t *path = p.path + (int64_t)b * W;
    const bool sound = lo >= 0 && lo <= hi && hi <= p.rows && !(tree && hi - lo > kMaxTree);
    if (!sound || lo == hi) {  // the whole cluster
        if (first) {
            for (int j = tid; j < W; j += kThreads) {
                tokens[j] = -1;
                path[j] = -1;
            }
            if (tid == 0) {
                p.lengths[b] = 0;
                if (!sound) atomicOr(p.watchdog, kv::kWatchIndex);
            }
        }
        cluster_wait();
        return;
    }
    const int64_t left = hi - lo;
    const int n = left > INT32_MAX ? INT32_MAX : (int)left;
    const T *probs = static_cast<const T *>(p.p) + lo * p.ldp;
    const T *drafts = p.q ? static_cast<const T *>(p.q) + lo * p.ldq : nullptr;
    auto token_of = [&](int row) -> int {  // -1: outside the vocabulary
        const int64_t x = p.tokens[lo + row];
        return x >= 0 && x < p.V ? (int)x : -1;
    };
    bool bad = false;
    int length, last;
    bool refused;  // whether tokens drafted below the last accepted row were refused
    if (!tree) {
        // the first refusal, its last bit whether a token was refused (what is none takes
        // nothing); rows from W on are not looked at
        const int most = min(n, W);
        if (tid == 0) s_stop = 2 * most;
        __syncthreads();
        for (int r = 1 + tid; r < most; r += kThreads) {
            const int x = token_of(r);
            bool ok = false;
            if (r < kMaxTree) s_token[r] = x;
            if (x >= 0) {
                const float u = p.u[lo + r - 1], px = unit(DT<T>::to_f(probs[(r - 1) * p.ldp + x]));
                if (drafts)  // exact in binary64
                    ok = (double)u * (double)unit(DT<T>::to_f(drafts[r * p.ldq + x])) < (double)px;
                else
                    ok = fixed(u) < fixed(px);
            }
            bad |= x < 0;
            if (!ok) atomicMin(&s_stop, 2 * r + (x >= 0));
        }
        __syncthreads();
        length = s_stop >> 1;
        last = length - 1;
        refused = s_stop & 1;
    } else {
        for (int r = tid; r < n; r += kThreads) {
            int up = -1, x = -1;
            int64_t mass = 0;
            if (r > 0) {
                up = p.parents[lo + r];
                x = token_of(r);
                if (up < 0 || up >= r || x < 0) {
                    bad = true;
                    up = -1;  // no one's child
                } else {
                    mass = fixed(DT<T>::to_f(probs[up * p.ldp + x]));
                }
            }
            s_parent[r] = up;
            s_token[r] = x;
            s_mass[r] = mass;
            s_next[r] = -1;
            s_u[r] = fixed(p.u[lo + r]);
        }
        __syncthreads();
        for (int r = 1 + tid; r < n; r += kThreads) {
            const int up = s_parent[r];
            if (up < 0) continue;
            bool again = false;
            for (int s = up + 1; s < r; ++s) again |= s_parent[s] == up && s_token[s] == s_token[r];
            if (again) s_mass[r] = 0;
        }
        __syncthreads();
        for (int r = 1 + tid; r < n; r += kThreads) {
            const int up = s_parent[r];
            if (up < 0) continue;
            int64_t low = 0;
            for (int s = up + 1; s < r; ++s)
                if (s_parent[s] == up) low += s_mass[s];
            const int64_t u = s_u[up];
            if (low <= u && u < low + s_mass[r]) s_next[up] = r;  // one child at most
        }
        __syncthreads();
        if (tid == 0) {
            int at = 0, m = 0;
            s_walk[m++] = 0;
            while (m < W && s_next[at] >= 0) s_walk[m++] = at = s_next[at];
            s_length = m;
            s_deep = m < W;
        }
        __syncthreads();
        length = s_length;
        last = s_walk[length - 1];
        refused = s_deep;  // the children of `last`, if any
    }
    if (first) {
        if (bad) atomicOr(p.watchdog, kv::kWatchIndex);
        for (int j = tid; j < W; j += kThreads) {
            path[j] = j < length ? (tree ? s_walk[j] : j) : -1;
            if (j < length - 1) {
                const int r = tree ? s_walk[j + 1] : j + 1;
                tokens[j] = r < kMaxTree ? s_token[r] : p.tokens[lo + r];
            } else if (j >= length) {
                tokens[j] = -1;
            }
        }
        if (tid == 0) p.lengths[b] = length;
    }

    // the draw
    const T *pr = probs + last * p.ldp;
    int mode = !refused ? W_ALL : drafts ? W_REST : W_WITHOUT;
    const T *qr = mode == W_REST ? drafts + (last + 1) * p.ldq : pr;
    const float v = fminf(unit(p.v[b]), 0.99999994f);
    // the refused children's tokens, in s_next
    if (tid == 0) s_gone = 0;
    __syncthreads();
    if (mode == W_WITHOUT) {
        auto refuse = [&](int x) { s_next[atomicAdd(&s_gone, 1)] = x; };
        if (tree) {
            for (int s = last + 1 + tid; s < n; s += kThreads)
                if (s_parent[s] == last && s_mass[s] > 0) refuse(s_token[s]);
        } else if (tid == 0) {  // a chain's only child
            refuse(last + 1 < kMaxTree ? s_token[last + 1] : token_of(last + 1));
        }
    }
    __syncthreads();
    const int groups = (p.V + kGroup - 1) / kGroup;
    const int g0 = (int)((int64_t)groups * rank / cluster);
    const int g1 = (int)((int64_t)groups * (rank + 1) / cluster);
    constexpr int64_t kTooMuch = int64_t(2) << kFrac;  // no distribution
    cluster_wait();
    for (int turn = 0;; ++turn) {
        for (int g = g0 + (tid >> 5); g < g1; g += kWarps) {
            const int64_t s = mode == W_REST ? group_sum64<T, true>(pr, qr, g, p.V, p.vec)
                                             : group_sum64<T, false>(pr, pr, g, p.V, p.vec);
            if ((tid & 31) == 0) s_group[g - g0] = s;
        }
        __syncthreads();
        if (mode == W_WITHOUT) {  // each of them once
            for (int i = tid; i < s_gone; i += kThreads) {
                const int x = s_next[i], g = x / kGroup;
                if (g >= g0 && g < g1)
                    atomicAdd(reinterpret_cast<unsigned long long *>(&s_group[g - g0]),
                              (unsigned long long)-fixed(DT<T>::to_f(pr[x])));
            }
            __syncthreads();
        }
        // this CTA's groups, four to a thread, clamped so that no sum of theirs overflows
        constexpr int kEach = kMaxGroups / kThreads;
        int64_t mine = 0, total;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int g = tid * kEach + i;
            if (g < g1 - g0) mine += min(s_group[g], kTooMuch);
        }
        const int64_t before = block_scan64(mine, red, &total);
        if (tid < cluster) store_peer(&s_part[turn][rank], tid, total);
        cluster_arrive();
        cluster_wait();
        int64_t ahead = 0, all = 0;
        for (int r = 0; r < cluster; ++r) {
            if (r == rank) ahead = all;
            all += s_part[turn][r];
        }
        if (all == 0 && mode != W_ALL) {  // nothing left: the cluster as one
            mode = W_ALL;
            continue;
        }
        if (all == 0 || all >= kTooMuch) {
            if (first && tid == 0) {
                tokens[length - 1] = -1;
                atomicOr(p.watchdog, kv::kWatchIndex);
            }
            return;
        }
        // the whole part: the product has up to 71 bits, rounded down as the cut is
        const int64_t target = (int64_t)__dmul_rd((double)v, (double)all) - ahead;
        if (target < 0 || target >= total) return;  // another CTA's
        if (target >= before && target < before + mine) {
            int64_t sum = before;
            int found = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int g = tid * kEach + i;
                if (g < g1 - g0) {
                    const int64_t w = s_group[g];
                    if (sum <= target && target < sum + w) {
                        found = g;
                        s_mass[0] = sum;  // its rows are no longer needed
                    }
                    sum += w;
                }
            }
            s_found = found;
        }
        __syncthreads();
        // inside the group: neighbouring elements to a thread
        constexpr int kMine = kGroup / kThreads;
        const int x0 = (g0 + s_found) * kGroup + tid * kMine;
        const int64_t rest = target - s_mass[0];
        int64_t w[kMine], own = 0, ignored;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int x = x0 + i;
            w[i] = 0;
            if (x < p.V) {
                w[i] = weight(DT<T>::to_f(pr[x]), mode == W_REST ? DT<T>::to_f(qr[x]) : 0.f,
                              mode == W_REST);
            }
        }
        if (mode == W_WITHOUT) {
            for (int k = 0; k < s_gone; ++k) {
                const int i = s_next[k] - x0;
#pragma unroll
                for (int m = 0; m < kMine; ++m)
                    if (i == m) w[m] = 0;
            }
        }
#pragma unroll
        for (int i = 0; i < kMine; ++i) own += w[i];
        int64_t sum = block_scan64(own, red, &ignored);
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            if (sum <= rest && rest < sum + w[i]) tokens[length - 1] = x0 + i;
            sum += w[i];
        }
        return;
    }
}

// Host launcher (instantiated per storage type).
template <typename T>
cudaError_t launch_verify(const Params &p, int num_sms, bool pdl, cudaStream_t st);

}  // namespace verify
}  // namespace rarn
