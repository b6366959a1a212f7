// A team of warps on the rows of a slab: the pieces that both directions of the block norms share.
//
// A thread owns the same C = 4 or 8 columns of every row. Rows come through a ring of shared-memory
// stages filled by cp.async; rows too long for 16 warps are split over a cluster of 2, 4 or 8 CTAs,
// whose warps exchange their sums through distributed shared memory.
//
// Two layouts of a row over the threads:
// * aligned rows (every row of every matrix starts on 16 bytes): slot s of thread t is the
//   16 bytes s x team + t; a thread reads back what it copied itself, so no barrier;
// * other rows: the 16-byte granules that cover the row are copied as they lie, the
//   team meets at a barrier, and element k of thread t is column k x team + t, which any phase
//   reads and writes without bank conflicts or partial sectors.
#pragma once

#include <algorithm>
#include <initializer_list>

#include "tr_block.cuh"
#include "tr_block.h"
#include "tr_launch.h"

namespace tr {
namespace block {

constexpr int kMaxWarps = 16;   // of a team in one CTA
constexpr int kMaxCluster = 8;

// How a launch maps rows onto threads and shared memory.
struct RowShape {
    int warps;         // a team's in one CTA
    int teams;         // of a CTA
    int cluster;       // CTAs of a row
    int cta_vecs;      // 16-byte slots of a row in one CTA
    int stages;        // of a team's ring, 3 or 4: two rows are at work, the others on their way
    int tensors;       // matrices read
    int tensor_bytes;  // shared memory of one matrix's row
};

// Shared memory of a team's exchanges (up to four values): for each warp of a row two halves of 8 floats, its
// columns and their reciprocal; of all teams; and of the whole CTA.
__host__ __device__ inline int team_bytes(const RowShape& g) { return (2 * 8 + 2) * 4 * g.warps * g.cluster; }
__host__ __device__ inline int fixed_bytes(const RowShape& g) { return (g.teams * team_bytes(g) + 127) / 128 * 128; }
inline int row_smem(const RowShape& g) { return fixed_bytes(g) + g.teams * g.stages * g.tensors * g.tensor_bytes; }

// Wait for a row of a ring of 3 or 4 stages whose copies were begun `newer` (1 or 2, for 3 stages) rows ago or
// earlier; with 4 stages one more row stays under way.
__device__ __forceinline__ void ring_wait(int stages, int newer) {
    if (stages == 3) newer == 1 ? cp_async_wait<0>() : cp_async_wait<1>();
    else newer == 1 ? cp_async_wait<1>() : cp_async_wait<2>();
}

// N values summed over the lanes below 2 x BIT, in one halving step per bit of the value's index
// (N/2 + N/4 + ... + the other bits: 6 shuffles for 4 values over a warp, not 20). The lanes
// whose upper bits are i end with value i.
template <int N, int BIT>
__device__ __forceinline__ float halving_sums(const float (&v)[N], int lane) {
    if constexpr (N == 1) {
        float r = v[0];
#pragma unroll
        for (int o = BIT; o >= 1; o >>= 1) r += __shfl_xor_sync(kFull, r, o);
        return r;
    } else {
        const bool up = lane & BIT;
        float o[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float keep = up ? v[i + N / 2] : v[i], send = up ? v[i] : v[i + N / 2];
            o[i] = keep + __shfl_xor_sync(kFull, send, BIT);
        }
        return halving_sums<N / 2, BIT / 2>(o, lane);
    }
}

// One team's exchange: N (2 or 4) sums over all warps of a row.
template <bool CLUSTER, int N>
struct Exchange {
    static constexpr int kLanes = 32 / N;  // lanes of a warp that end with the same value
    float* slot;   // this CTA's: 2 x 2 N x entries floats, then the entries' column counts
    int entries;   // warps of the row
    int entry;     // this warp's place among them
    int team, warps;
    int buf = 0;

    // this warp's value i (held by lanes kLanes i ..) into place `at + i` of its entry, in every CTA
    __device__ __forceinline__ void put(float r, int at, int stride) {
        const int lane = threadIdx.x & 31, l = lane % kLanes;
        float* s = slot + buf * 2 * N * entries + entry * stride + at + lane / kLanes;
        if constexpr (CLUSTER) {  // the lanes of a value (8 or more) store it to a CTA each
            cg::cluster_group cl = cg::this_cluster();
            if (l < static_cast<int>(cl.num_blocks())) *cl.map_shared_rank(s, l) = r;
        } else {
            if (l == 0) *s = r;
        }
    }
    __device__ __forceinline__ const float* meet() {
        if constexpr (CLUSTER) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        else team_barrier(team, warps);
        const float* s = slot + buf * 2 * N * entries;
        buf ^= 1;  // (the other half is free: every warp has read it before it came to this barrier)
        return s;
    }
    static __device__ __forceinline__ void spread(float r, float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(kFull, r, kLanes * i);
    }
    // f(entry) for this lane's entries: `per` lanes take one each at a time (a CTA's warps are at most 16)
    template <class F>
    __device__ __forceinline__ void each(int first, int per, F&& f) const {
        if constexpr (CLUSTER) {
            for (int e = first; e < entries; e += per) f(e);
        } else {
            if (first < entries) f(first);
        }
    }

    // v summed over the row
    __device__ __forceinline__ void sums(float (&v)[N]) {
        const int lane = threadIdx.x & 31;
        float r = halving_sums<N, 16>(v, lane);
        if (!CLUSTER && entries == 1) return spread(r, v);
        put(r, 0, N);
        const float* s = meet() + (lane >> 4) * (N / 2);
        float t[N / 2] = {};  // half the values a lane
        each(lane & 15, 16, [&](int e) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) t[i] += s[e * N + i];
        });
        spread(halving_sums<N / 2, 8>(t, lane), v);
    }

    // LayerNorm's sums. v: the thread's plain sums; about(means, w): given the warp's own means of the first
    // CENTRED values, the thread's sums w of squares and products about them. At the end v holds the row's
    // sums. w[i] are moved from the warps' means to the row's by shift(i, n, d, sums): what value i of an entry
    // of n columns gains when its means are d from the row's.
    template <int CENTRED, class A, class S>
    __device__ __forceinline__ void moments(float (&v)[N], float (&w)[N], float inv_n, A&& about, S&& shift) {
        const int lane = threadIdx.x & 31;
        const float* counts = slot + 4 * N * entries;  // columns, and their reciprocals
        const float r = halving_sums<N, 16>(v, lane);
        float m[CENTRED];
        const float inv = counts[entries + entry];
#pragma unroll
        for (int i = 0; i < CENTRED; ++i) m[i] = __shfl_sync(kFull, r, kLanes * i) * inv;
        about(m, w);
        const float rw = halving_sums<N, 16>(w, lane);
        if (!CLUSTER && entries == 1) {
            spread(r, v);
            spread(rw, w);
            return;
        }
        put(r, 0, 2 * N);
        put(rw, N, 2 * N);
        const float* s = meet();
        float q[N] = {}, t[N] = {};
        each(lane, 32, [&](int e) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                q[i] = s[e * 2 * N + i];
                t[i] += q[i];
            }
        });
        spread(halving_sums<N, 16>(t, lane), v);
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = 0.0f;
        each(lane, 32, [&](int e) {
            if constexpr (CLUSTER)
#pragma unroll
                for (int i = 0; i < N; ++i) q[i] = s[e * 2 * N + i];
            const float n = counts[e], rn = counts[entries + e];
            float d[CENTRED];
#pragma unroll
            for (int i = 0; i < CENTRED; ++i) d[i] = fmaf(q[i], rn, -v[i] * inv_n);
#pragma unroll
            for (int i = 0; i < N; ++i) t[i] += s[e * 2 * N + N + i] + shift(i, n, d, q);
        });
        spread(halving_sums<N, 16>(t, lane), w);
    }
    // The entries' column counts for moments().
    template <int S, int E, bool ODD>
    __device__ __forceinline__ void count_columns(int cols, int cta_vecs, int t) {
        float* counts = slot + 4 * N * entries;
        for (int e = t; e < entries; e += warps * 32) {
            const int there = min(cols - e / warps * cta_vecs * E, cta_vecs * E);
            int n = 0;
            for (int k = 0; k < (ODD ? S * E : S); ++k) {
                const int left = (ODD ? there : there / E) - (e % warps * 32 + warps * 32 * k);
                n += max(0, min(32, left)) * (ODD ? 1 : E);
            }
            counts[e] = static_cast<float>(n);  // (0: a warp past the end of the row's last part)
            counts[entries + e] = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
        }
        team_barrier(team, warps);
    }
};

// A pair of adjacent elements of a type.
__device__ __forceinline__ float2 pair_of(uint32_t q, __nv_bfloat16) {
    return make_float2(__uint_as_float(q << 16), __uint_as_float(q & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_of(uint32_t q, __half) {
    return __half22float2(*reinterpret_cast<const __half2*>(&q));
}
__device__ __forceinline__ uint32_t bits_of(float2 v, __nv_bfloat16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint32_t bits_of(float2 v, __half) {
    const __half2 b = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// A thread's share of a row, in one of the two layouts. `mine` columns of the row, from byte `base`
// on, belong to this CTA.
template <class T, int S, bool ODD>
struct Lanes {
    static constexpr int E = 16 / static_cast<int>(sizeof(T));  // elements of a slot
    static constexpr int P = E / 2;                             // pairs
    int t, tt;   // thread of the team, and its threads
    int mine, vecs;
    int64_t row_bytes, base;

    __device__ __forceinline__ Lanes(int t_, int tt_, int cols, int col0, int cta_vecs)
        : t(t_), tt(tt_), mine(min(cols - col0, cta_vecs * E)), vecs(mine / E),
          row_bytes(static_cast<int64_t>(cols) * static_cast<int>(sizeof(T))),
          base(static_cast<int64_t>(col0) * static_cast<int>(sizeof(T))) {}

    // column (of this CTA) of element e of slot s, and whether it is in the row
    __device__ __forceinline__ int column(int s, int e) const { return ODD ? t + tt * (s * E + e) : (t + tt * s) * E + e; }
    __device__ __forceinline__ bool in(int s, int e) const { return ODD ? column(s, e) < mine : t + tt * s < vecs; }
    // f(pair, are its elements in the row) for the pairs of slot s that are (in part) in the row
    template <class F>
    __device__ __forceinline__ void pairs(int s, F&& f) const {
        if constexpr (ODD) {
#pragma unroll
            for (int j = 0; j < P; ++j) f(j, in(s, 2 * j), in(s, 2 * j + 1));
        } else {
            if (in(s, 0))
#pragma unroll
                for (int j = 0; j < P; ++j) f(j, true, true);
        }
    }

    // start copying this CTA's part of a row to shared memory
    __device__ __forceinline__ void fetch(const void* matrix, int64_t rows, int64_t row, char* to) const {
        const char* from = static_cast<const char*>(matrix) + (row * row_bytes + base);
        if constexpr (!ODD) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int k = t + tt * s;
                if (k < vecs) cp_async16(smem_addr(to) + k * 16, from + k * 16);
            }
        } else {
            const int phase = static_cast<int>(reinterpret_cast<uintptr_t>(from) & 15);
            const int granules = (phase + mine * static_cast<int>(sizeof(T)) + 15) >> 4;
            const char* lo = static_cast<const char*>(matrix);
            const char* hi = lo + rows * row_bytes;
            for (int k = t; k < granules; k += tt) {
                const char* q = from - phase + k * 16;
                if (q >= lo && q + 16 <= hi) {
                    cp_async16(smem_addr(to) + k * 16, q);
                } else {  // the matrix's own first or last granule: its elements alone
                    for (int e = 0; e < E; ++e) {
                        const char* qe = q + e * static_cast<int>(sizeof(T));
                        if (qe >= lo && qe < hi) reinterpret_cast<T*>(to)[k * E + e] = *reinterpret_cast<const T*>(qe);
                    }
                }
            }
        }
    }
    // the pairs of slot s of the row staged at m; 0 outside the row
    __device__ __forceinline__ void load(const char* m, const void* matrix, int64_t row, int s, float2 (&v)[P]) const {
        if constexpr (!ODD) {
            uint4 q = make_uint4(0, 0, 0, 0);
            if (t + tt * s < vecs) q = *reinterpret_cast<const uint4*>(m + (t + tt * s) * 16);
            if constexpr (sizeof(T) == 4) {
                v[0] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
                v[1] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
            } else {
                v[0] = pair_of(q.x, T());
                v[1] = pair_of(q.y, T());
                v[2 % P] = pair_of(q.z, T());
                v[3 % P] = pair_of(q.w, T());
            }
        } else {
            const int phase = static_cast<int>((reinterpret_cast<uintptr_t>(matrix) + (row * row_bytes + base)) & 15);
            const T* e = reinterpret_cast<const T*>(m + phase);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                v[j].x = in(s, 2 * j) ? to_float(e[column(s, 2 * j)]) : 0.0f;
                v[j].y = in(s, 2 * j + 1) ? to_float(e[column(s, 2 * j + 1)]) : 0.0f;
            }
        }
    }
    __device__ __forceinline__ void store(void* out, int64_t row, int s, const float2 (&v)[P]) const {
        char* to = static_cast<char*>(out) + (row * row_bytes + base);
        if constexpr (!ODD) {
            if (t + tt * s < vecs) {
                uint4 q;
                if constexpr (sizeof(T) == 4) {
                    q = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
                } else {
                    q = make_uint4(bits_of(v[0], T()), bits_of(v[1], T()), bits_of(v[2 % P], T()), bits_of(v[3 % P], T()));
                }
                *reinterpret_cast<uint4*>(to + (t + tt * s) * 16) = q;
            }
        } else {
            T* o = reinterpret_cast<T*>(to);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                if (in(s, 2 * j)) o[column(s, 2 * j)] = from_float<T>(v[j].x);
                if (in(s, 2 * j + 1)) o[column(s, 2 * j + 1)] = from_float<T>(v[j].y);
            }
        }
    }
    // a parameter vector (from this CTA's first column on) at slot s's columns
    __device__ __forceinline__ void param(const float* w, int s, float absent, float2 (&v)[P]) const {
#pragma unroll
        for (int j = 0; j < P; ++j) v[j] = both(absent);
        if (!w) return;
        if (!ODD && aligned16(w)) {
            if (t + tt * s < vecs)
#pragma unroll
                for (int j = 0; j < P; j += 2) {
                    const float4 q = ld_param4(w + column(s, 2 * j));
                    v[j] = make_float2(q.x, q.y);
                    v[j + 1] = make_float2(q.z, q.w);
                }
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                if (in(s, 2 * j)) v[j].x = __ldg(w + column(s, 2 * j));
                if (in(s, 2 * j + 1)) v[j].y = __ldg(w + column(s, 2 * j + 1));
            }
        }
    }
};

// ---- host side -------------------------------------------------------------

// The layout of a pass over `tensors` matrices, or warps = 0 when a row does not fit: 8 columns
// a thread at most, the fewest CTAs a row that this allows with three stages of ring (four where
// they leave `ctas` CTAs an SM), and several teams in a CTA for short rows.
template <class T>
RowShape row_shape(int cols, int tensors, bool odd, int ctas, int* slots) {
    constexpr int E = 16 / static_cast<int>(sizeof(T));
    constexpr int kMaxSlots = 8 / E;
    constexpr int kLimit = 226 * 1024;
    RowShape g = {};
    const int vecs = (cols + E - 1) / E;
    for (g.cluster = 1; g.cluster <= kMaxCluster; g.cluster *= 2) {
        g.cta_vecs = (vecs + g.cluster - 1) / g.cluster;
        const int s = (g.cta_vecs + 32 * kMaxWarps - 1) / (32 * kMaxWarps);
        if (s > kMaxSlots) continue;
        *slots = s;
        g.warps = (g.cta_vecs + 32 * s - 1) / (32 * s);
        g.teams = g.cluster > 1 ? 1 : std::max(1, 8 / g.warps);
        g.tensors = tensors;
        g.tensor_bytes = g.cta_vecs * 16 + (odd ? 16 : 0);
        g.stages = 4;
        if (ctas * (row_smem(g) + 1024) > kLimit) g.stages = 3;
        if (row_smem(g) <= kLimit) return g;
    }
    g.warps = 0;
    return g;
}

// Whether every row of these matrices starts and ends on 16 bytes.
inline bool rows_aligned(int64_t row_bytes, std::initializer_list<const void*> matrices) {
    bool ok = row_bytes % 16 == 0;
    for (const void* m : matrices) ok = ok && reinterpret_cast<uintptr_t>(m) % 16 == 0;
    return ok;
}

}  // namespace block
}  // namespace tr
