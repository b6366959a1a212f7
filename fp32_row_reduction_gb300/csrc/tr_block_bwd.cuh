// The gated residual norm's backward with the rows on chip (see k_block_bwd.cu for
// the formulas).
//
// HBM-bound: h, a, dy and dh are read and dx and da written once. A team of warps
// takes a row at a time; a thread owns the same C = 4 or 8 columns of every row of its
// slab, so the column sums stay in its registers (32-bit) until the slab ends. Rows come through a
// ring of shared-memory stages filled by cp.async. Rows too long for 16 warps are split
// over a cluster of 2, 4 or 8 CTAs.
//
// With 16-bit types the work per byte is what limits: at 4096 columns a SM has 2090 cycles to
// the row. So the arithmetic is on pairs (f32x2), which norms there are is known when the kernel is
// compiled, and there is one exchange between warps a row: the next row's statistics travel with
// this row's sum of q ah. LayerNorm's squares are taken about the warp's own mean and moved to the
// row's when the warps meet (Chan, Golub and LeVeque 1979), so it needs no second exchange.
//
// Two layouts of a row over the threads:
// * aligned rows (every row of every matrix starts on 16 bytes): slot s of thread t is the
//   16 bytes s x team + t; a thread reads back what it copied itself, so no barrier;
// * other rows: the 16-byte granules that cover the row are copied as they lie, the
//   team meets at a barrier, and element k of thread t is column k x team + t, which any phase
//   reads and writes without bank conflicts or partial sectors.
#pragma once

#include <algorithm>

#include "tr_block.cuh"
#include "tr_block.h"
#include "tr_launch.h"

namespace tr {
namespace block {

constexpr int kBwMaxWarps = 16;
constexpr int kBwMaxStages = 4;
constexpr int kBwMaxCluster = 8;

// How a launch maps rows onto threads and shared memory.
struct BwShape {
    int warps;         // a team's in one CTA
    int teams;         // of a CTA
    int cluster;       // CTAs of a row
    int cta_vecs;      // 16-byte slots of a row in one CTA
    int stages;        // of a team's ring (3 or more: two rows are at work, the others on their way)
    int tensors;       // matrices read
    int tensor_bytes;  // shared memory of one matrix's row
};

// Shared memory of the teams' exchanges: for each warp of a row two halves of 8 floats, and its columns.
__host__ __device__ inline int bwd_team_bytes(const BwShape& g) { return (2 * 8 + 4) * 4 * g.warps * g.cluster; }
__host__ __device__ inline int bwd_fixed_bytes(const BwShape& g) { return (g.teams * bwd_team_bytes(g) + 127) / 128 * 128; }

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

// One team's exchange: sums over all warps of a row.
template <bool CLUSTER>
struct Exchange {
    float* slot;   // this CTA's: 2 x 8 x entries floats, then the entries' column counts
    int entries;   // warps of the row
    int entry;     // this warp's place among them
    int team, warps;
    int buf = 0;

    // this warp's value i (held by lanes 8 i ..) into place `at + i` of its entry, in every CTA
    __device__ __forceinline__ void put(float r, int at, int stride) {
        const int lane = threadIdx.x & 31;
        float* s = slot + buf * 8 * entries + entry * stride + at + (lane >> 3);
        if constexpr (CLUSTER) {  // the eight lanes of a value store it to a CTA each
            cg::cluster_group cl = cg::this_cluster();
            if ((lane & 7) < static_cast<int>(cl.num_blocks())) *cl.map_shared_rank(s, lane & 7) = r;
        } else {
            if ((lane & 7) == 0) *s = r;
        }
    }
    __device__ __forceinline__ const float* meet() {
        if constexpr (CLUSTER) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        else team_barrier(team, warps);
        const float* s = slot + buf * 8 * entries;
        buf ^= 1;  // (the other half is free: every warp has read it before it came to this barrier)
        return s;
    }
    static __device__ __forceinline__ void spread(float r, float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(kFull, r, 8 * i);
    }

    // v summed over the row
    __device__ __forceinline__ void sums(float (&v)[4]) {
        const int lane = threadIdx.x & 31;
        float r = halving_sums<4, 16>(v, lane);
        if (!CLUSTER && entries == 1) return spread(r, v);
        put(r, 0, 4);
        const float* s = meet();
        float t[2] = {0.0f, 0.0f};  // 16 entries at a time, two values a lane
        for (int e = lane & 15; e < entries; e += 16) {
            const float2 q = *reinterpret_cast<const float2*>(s + e * 4 + (lane >> 4) * 2);
            t[0] += q.x;
            t[1] += q.y;
        }
        spread(halving_sums<2, 8>(t, lane), v);
    }

    // The warp's sums of h, a and u, and of q (v); then about(mean h, mean a, w), which gives the sums of
    // squares and products about those means of the warp's own columns in w[0 .. 2] (w[3]: as it is). At the end v holds
    // the row's sums and w those about the row's means.
    template <class F>
    __device__ __forceinline__ void moments(float (&v)[4], float (&w)[4], float inv_n, F&& about) {
        const int lane = threadIdx.x & 31;
        float* counts = slot + 16 * entries;
        const float r = halving_sums<4, 16>(v, lane);
        const float inv = 1.0f / counts[entry];
        about(__shfl_sync(kFull, r, 0) * inv, __shfl_sync(kFull, r, 8) * inv, w);
        const float rw = halving_sums<4, 16>(w, lane);
        if (!CLUSTER && entries == 1) {
            spread(r, v);
            spread(rw, w);
            return;
        }
        put(r, 0, 8);
        put(rw, 4, 8);
        const float* s = meet();
        float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int e = lane; e < entries; e += 32) {
            const float4 q = *reinterpret_cast<const float4*>(s + e * 8);
            t[0] += q.x;
            t[1] += q.y;
            t[2] += q.z;
            t[3] += q.w;
        }
        spread(halving_sums<4, 16>(t, lane), v);
        const float mh = v[0] * inv_n, ma = v[1] * inv_n;
        t[0] = t[1] = t[2] = t[3] = 0.0f;
        for (int e = lane; e < entries; e += 32) {
            const float4 q = *reinterpret_cast<const float4*>(s + e * 8), z = *reinterpret_cast<const float4*>(s + e * 8 + 4);
            const float n = counts[e];
            const float dh = q.x / n - mh, da = q.y / n - ma;  // the entry's means about the row's
            t[0] += fmaf(n * dh, dh, z.x);
            t[1] += fmaf(n * da, da, z.y);
            t[2] += fmaf(dh, q.z, z.z);
            t[3] += z.w;
        }
        spread(halving_sums<4, 16>(t, lane), w);
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

// MODE: the norms there are, a mask of TR_BLOCK_POST and TR_BLOCK_PRE; 0: as p says.
template <class T, bool LAYER, int S, bool ODD, bool CLUSTER, int MODE, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) bwd_kernel(const BlockBwArgs p, const BwShape g) {
    constexpr int E = 16 / static_cast<int>(sizeof(T));
    constexpr int P = E / 2;       // pairs of a slot
    constexpr int K = S * P;       // pairs of a thread
    constexpr int V = LAYER ? 4 : 2;
    const bool pre = MODE ? (MODE & TR_BLOCK_PRE) != 0 : p.pre != 0;
    const bool post = MODE ? (MODE & TR_BLOCK_POST) != 0 : p.post != 0;
    extern __shared__ uint4 smem[];
    const int tt = g.warps * 32;  // a team's threads in this CTA
    const int team = CLUSTER ? 0 : static_cast<int>(threadIdx.x) / tt;
    const int t = static_cast<int>(threadIdx.x) - team * tt;
    const int rank = CLUSTER ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
    const int cols = p.cols;
    const int col0 = rank * g.cta_vecs * E;                 // this CTA's first column
    const int mine = min(cols - col0, g.cta_vecs * E);      // and how many it has
    const int vecs = mine / E;                              // aligned rows: 16-byte slots
    const float inv_n = 1.0f / static_cast<float>(cols);
    Exchange<CLUSTER> ex{reinterpret_cast<float*>(smem) + team * (bwd_team_bytes(g) / 4), g.warps * g.cluster,
                         rank * g.warps + (t >> 5), team, g.warps};
    const int stage_bytes = g.tensors * g.tensor_bytes;
    char* ring = reinterpret_cast<char*>(smem) + bwd_fixed_bytes(g) + team * g.stages * stage_bytes;
    if constexpr (LAYER) {  // the columns of each warp of the row
        float* counts = ex.slot + 16 * ex.entries;
        for (int e = t; e < ex.entries; e += tt) {
            const int first = e / g.warps * g.cta_vecs * E, there = min(cols - first, g.cta_vecs * E);
            int n = 0;
            for (int k = 0; k < (ODD ? S * E : S); ++k) {
                const int left = (ODD ? there : there / E) - (e % g.warps * 32 + tt * k);
                n += max(0, min(32, left)) * (ODD ? 1 : E);
            }
            counts[e] = static_cast<float>(max(1, n));
        }
        team_barrier(team, g.warps);
    }
    if constexpr (CLUSTER) cg::this_cluster().sync();  // every CTA of the cluster runs before it is written to
    pdl_enter();

    // column (of this CTA) of element e of slot s
    auto column = [&](int s, int e) { return ODD ? t + tt * (s * E + e) : (t + tt * s) * E + e; };
    // whether slot s (pair j of it, in the odd layout element by element) is inside the row
    auto in = [&](int s, int e) { return ODD ? column(s, e) < mine : t + tt * s < vecs; };

    const int64_t index = CLUSTER ? blockIdx.x / g.cluster : static_cast<int64_t>(blockIdx.x) * g.teams + team;
    if (index >= p.slabs) return;  // (a whole cluster, or a whole team)
    const SlabRows slab = slab_rows(p, index);

    // ---- the ring: h and dy (pre), a, dh, each where there is one ----
    const bool need_a = post || p.dgate;
    const int at_dy = pre ? g.tensor_bytes : 0;
    const int at_a = pre ? 2 * g.tensor_bytes : 0;
    const int at_dh = at_a + (need_a ? g.tensor_bytes : 0);
    const int64_t row_bytes = static_cast<int64_t>(cols) * static_cast<int>(sizeof(T));
    const int64_t base = static_cast<int64_t>(col0) * static_cast<int>(sizeof(T));
    auto fetch_one = [&](const void* matrix, int64_t row, char* to) {
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
            const char* hi = lo + p.rows * row_bytes;
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
    };
    auto fetch = [&](int64_t row, int stage) {
        if (row < slab.end) {
            char* to = ring + stage * stage_bytes;
            if (pre) {
                fetch_one(p.h, row, to);
                fetch_one(p.dy, row, to + at_dy);
            }
            if (need_a) fetch_one(p.a, row, to + at_a);
            if (p.dh) fetch_one(p.dh, row, to + at_dh);
        }
        cp_async_commit();
    };
    // the pairs of slot s of the matrix staged at `m`; 0 outside the row
    auto load = [&](const char* m, const void* matrix, int64_t row, int s, float2 (&v)[P]) {
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
    };
    auto store = [&](void* out, int64_t row, int s, const float2 (&v)[P]) {
        if constexpr (!ODD) {
            if (t + tt * s < vecs) {
                uint4 q;
                if constexpr (sizeof(T) == 4) {
                    q = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
                } else {
                    q = make_uint4(bits_of(v[0], T()), bits_of(v[1], T()), bits_of(v[2 % P], T()), bits_of(v[3 % P], T()));
                }
                *reinterpret_cast<uint4*>(static_cast<char*>(out) + (row * row_bytes + base) + (t + tt * s) * 16) = q;
            }
        } else {
            T* o = static_cast<T*>(out) + row * cols + col0;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                if (in(s, 2 * j)) o[column(s, 2 * j)] = from_float<T>(v[j].x);
                if (in(s, 2 * j + 1)) o[column(s, 2 * j + 1)] = from_float<T>(v[j].y);
            }
        }
    };
    // a parameter vector (from this CTA's first column on) at slot s's columns
    auto param = [&](const float* w, int s, float absent, float2 (&v)[P]) {
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
    };
    auto at0 = [&](const float* w) { return w ? w + col0 : nullptr; };

    // the slab's column sums dy hh and dy; those of the running gate row, D ah and D
    float2 sum0[K], sumA[K], sum1[LAYER ? K : 1], sumB[LAYER ? K : 1];
    float2 w[K], qw[K];  // the pre-norm's weight; bs gate w_post
#pragma unroll
    for (int k = 0; k < K; ++k) {
        sum0[k] = sumA[k] = both(0.0f);
        if constexpr (LAYER) sum1[k] = sumB[k] = both(0.0f);
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        float2 v[P];
        param(pre ? at0(p.pre_w) : nullptr, s, 1.0f, v);
#pragma unroll
        for (int j = 0; j < P; ++j) w[s * P + j] = v[j];
    }
    auto gate_row = [&](int64_t row) { return p.gate ? p.gate + row / p.group_rows * cols + col0 : nullptr; };
    auto enter_group = [&](int64_t row) {
        const float* gr = gate_row(row);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float2 o[P], v[P];
            param(post ? at0(p.post_w) : nullptr, s, 1.0f, o);
            param(gr, s, 1.0f, v);
#pragma unroll
            for (int j = 0; j < P; ++j) qw[s * P + j] = __fmul2_rn(v[j], __fmul2_rn(both(p.bs), o[j]));
        }
    };
    // a whole group is done: its gate gradient is final, and its share of the post-norm's column
    // sums goes to the slab's partials, which no other thread touches
    bool flushed = false;
    auto leave_group = [&](int64_t row) {
        const float* gr = gate_row(row);
        float* dg = p.dgate ? p.dgate + row / p.group_rows * cols + col0 : nullptr;
        float* part = p.part + index * V * cols + col0;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float2 o[P], ob[P], gate[P];
            param(post ? at0(p.post_w) : nullptr, s, 1.0f, o);
            param(post ? at0(p.post_b) : nullptr, s, 0.0f, ob);
            param(gr, s, 1.0f, gate);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int k = s * P + j;
                auto one = [&](int c, float wt, float bias, float gt, float a, float b) {
                    if (dg) dg[c] = p.bs * (LAYER ? fmaf(wt, a, bias * b) : wt * a);
                    part[cols + c] = fmaf(gt, a, flushed ? part[cols + c] : 0.0f);
                    if constexpr (LAYER) part[3 * cols + c] = fmaf(gt, b, flushed ? part[3 * cols + c] : 0.0f);
                };
                const float2 b = LAYER ? sumB[LAYER ? k : 0] : both(0.0f);
                if (in(s, 2 * j)) one(column(s, 2 * j), o[j].x, ob[j].x, gate[j].x, sumA[k].x, b.x);
                if (in(s, 2 * j + 1)) one(column(s, 2 * j + 1), o[j].y, ob[j].y, gate[j].y, sumA[k].y, b.y);
                sumA[k] = both(0.0f);
                if constexpr (LAYER) sumB[k] = both(0.0f);
            }
        }
        flushed = true;
    };
    // f(pair, whether its elements are in the row) for the pairs of slot s that are (in part) in the row
    auto pairs = [&](int s, auto&& f) {
        if constexpr (ODD) {
#pragma unroll
            for (int j = 0; j < P; ++j) f(j, in(s, 2 * j), in(s, 2 * j + 1));
        } else {
            if (in(s, 0))
#pragma unroll
                for (int j = 0; j < P; ++j) f(j, true, true);
        }
    };
    auto about = [&](float2 v, float m, bool x_in, bool y_in) {  // v - m; 0 outside the row
        if constexpr (!LAYER) return v;
        float2 c = __fadd2_rn(v, both(-m));
        if (!x_in) c.x = 0.0f;
        if (!y_in) c.y = 0.0f;
        return c;
    };

    // ---- a row's statistics ----
    float mean_h = 0.0f, mean_a = 0.0f, c1 = 0.0f;  // LayerNorm: means of h, a, u
    // LayerNorm: the thread's sums of h, a and u
    auto plain_sums = [&](const char* m, int64_t row, float (&v)[4]) {
        float2 h2 = both(0.0f), a2 = both(0.0f), u2 = both(0.0f);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float2 x[P], y[P];
            if (pre) {
                load(m, p.h, row, s, x);
                load(m + at_dy, p.dy, row, s, y);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    h2 = __fadd2_rn(h2, x[j]);
                    u2 = __ffma2_rn(y[j], w[s * P + j], u2);
                }
            }
            if (post) {
                load(m + at_a, p.a, row, s, x);
#pragma unroll
                for (int j = 0; j < P; ++j) a2 = __fadd2_rn(a2, x[j]);
            }
        }
        v[0] = h2.x + h2.y;
        v[1] = a2.x + a2.y;
        v[2] = u2.x + u2.y;
    };
    // the thread's sums of (h - mh)^2, (a - ma)^2 and u (h - mh)
    auto square_sums = [&](const char* m, int64_t row, float mh, float ma, float (&v)[4]) {
        float2 h2 = both(0.0f), a2 = both(0.0f), u2 = both(0.0f);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float2 x[P], y[P];
            if (pre) {
                load(m, p.h, row, s, x);
                load(m + at_dy, p.dy, row, s, y);
                pairs(s, [&](int j, bool xi, bool yi) {
                    const float2 c = about(x[j], mh, xi, yi);
                    h2 = __ffma2_rn(c, c, h2);
                    u2 = __ffma2_rn(__fmul2_rn(y[j], w[s * P + j]), c, u2);
                });
            }
            if (post) {
                load(m + at_a, p.a, row, s, x);
                pairs(s, [&](int j, bool xi, bool yi) {
                    const float2 c = about(x[j], ma, xi, yi);
                    a2 = __ffma2_rn(c, c, a2);
                });
            }
        }
        v[0] = h2.x + h2.y;
        v[1] = a2.x + a2.y;
        v[2] = u2.x + u2.y;
    };
    // The statistics of row `row` staged at m (none when it is not there: `more` is false), with the sums of q
    // and q (a - mean) of the row before, which end in qs and qa. D = dh + r_h (u - c1 - (h - mean) k2) with
    // k2 = r_h^2 mean(u (h - mean)). rsqrtf is good to 2^-22, as the sums are.
    float rh = 0.0f, ra = 0.0f, k2 = 0.0f;
    auto statistics = [&](const char* m, int64_t row, bool more, float& qs, float& qa, auto&& between) {
        [[maybe_unused]] float v[4] = {0.0f, 0.0f, 0.0f, qs};
        float w4[4] = {0.0f, 0.0f, 0.0f, qa};
        if constexpr (LAYER) {
            if (more) plain_sums(m, row, v);
            ex.moments(v, w4, inv_n, [&](float mh, float ma, float (&o)[4]) {
                if (more) square_sums(m, row, mh, ma, o);
            });
            qs = v[3];
        } else {
            if (more) square_sums(m, row, 0.0f, 0.0f, w4);
            ex.sums(w4);
        }
        qa = w4[3];
        between();
        if constexpr (LAYER) {
            mean_h = v[0] * inv_n;
            mean_a = v[1] * inv_n;
            c1 = v[2] * inv_n;
        }
        if (pre) {
            rh = rsqrtf(fmaf(w4[0], inv_n, p.eps));
            k2 = w4[2] * inv_n * rh * rh;
        }
        if (post) ra = rsqrtf(fmaf(w4[1], inv_n, p.eps));
    };

    // ---- the first row ----
    // (the ring is three or four stages; a wait leaves the later rows' copies in flight)
    auto wait = [&](int newer) {
        if (g.stages == 3) newer == 1 ? cp_async_wait<0>() : cp_async_wait<1>();
        else newer == 1 ? cp_async_wait<1>() : cp_async_wait<2>();
    };
    auto odd_barrier = [&]() {
        if constexpr (CLUSTER) __syncthreads();
        else team_barrier(team, g.warps);
    };
    for (int i = 0; i + 1 < g.stages; ++i) fetch(slab.begin + i, i);
    wait(2);
    if constexpr (ODD) odd_barrier();
    {
        float qs = 0.0f, qa = 0.0f;
        statistics(ring, slab.begin, true, qs, qa, [] {});
    }

    int stage = 0, fill = g.stages - 1;
    int64_t left = 0;  // rows of the running group still to come
    for (int64_t row = slab.begin; row < slab.end; ++row) {
        if (left == 0) {
            enter_group(row);
            left = p.slices > 0 ? slab.end - slab.begin : p.group_rows;
        }
        if constexpr (ODD) {  // the next row is here, and every thread is done with the row before
            wait(1);
            odd_barrier();
        }
        fetch(row + g.stages - 1, fill);
        fill = fill + 1 == g.stages ? 0 : fill + 1;
        const char* m = ring + stage * stage_bytes;
        stage = stage + 1 == g.stages ? 0 : stage + 1;
        const char* next = ring + stage * stage_bytes;

        // D, dx, the column sums of the pre-norm, and the sums of q (a - mean) and q
        float2 d[K], av[K];
        float2 qa2 = both(0.0f), qs2 = both(0.0f);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float2 x[P], y[P], o[P];
            if (p.dh) {
                load(m + at_dh, p.dh, row, s, o);
            } else {
#pragma unroll
                for (int j = 0; j < P; ++j) o[j] = both(0.0f);
            }
            if (pre) {
                load(m, p.h, row, s, x);
                load(m + at_dy, p.dy, row, s, y);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const int k = s * P + j;
                    const float2 c = LAYER ? __fadd2_rn(x[j], both(-mean_h)) : x[j];
                    sum0[k] = __ffma2_rn(__fmul2_rn(y[j], both(rh)), c, sum0[k]);
                    if constexpr (LAYER) sum1[k] = __fadd2_rn(sum1[k], y[j]);
                    const float2 u = LAYER ? __ffma2_rn(y[j], w[k], both(-c1)) : __fmul2_rn(y[j], w[k]);
                    o[j] = __ffma2_rn(both(rh), __ffma2_rn(c, both(-k2), u), o[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < P; ++j) {
                d[s * P + j] = o[j];
                o[j] = __fmul2_rn(o[j], both(p.rs));
            }
            store(p.dx, row, s, o);
            if (need_a) {
                load(m + at_a, p.a, row, s, x);
#pragma unroll
                for (int j = 0; j < P; ++j) av[s * P + j] = LAYER && post ? __fadd2_rn(x[j], both(-mean_a)) : x[j];
                if (post)
                    pairs(s, [&](int j, bool xi, bool yi) {
                        float2 q = __fmul2_rn(d[s * P + j], qw[s * P + j]);
                        if (!xi) q.x = 0.0f;
                        if (!yi) q.y = 0.0f;
                        qa2 = __ffma2_rn(q, av[s * P + j], qa2);
                        if constexpr (LAYER) qs2 = __fadd2_rn(qs2, q);
                    });
            }
        }
        // the next row's statistics travel with this row's sums
        if constexpr (!ODD) wait(2);
        float qs = qs2.x + qs2.y, qa = qa2.x + qa2.y;
        statistics(next, row + 1, row + 1 < slab.end, qs, qa, [&] {
            // da, and the column sums of the post-norm and the gate
            const float e1 = qs * inv_n, e2 = qa * inv_n * ra * ra;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float2 o[P];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const int k = s * P + j;
                    float2 q = __fmul2_rn(d[k], qw[k]);
                    if (need_a) {
                        float2 ah = av[k];
                        if (post) {
                            q = __ffma2_rn(av[k], both(-e2), q);
                            if constexpr (LAYER) q = __fadd2_rn(q, both(-e1));
                            q = __fmul2_rn(q, both(ra));
                            ah = __fmul2_rn(av[k], both(ra));
                        }
                        sumA[k] = __ffma2_rn(d[k], ah, sumA[k]);
                        if constexpr (LAYER) sumB[k] = __fadd2_rn(sumB[k], d[k]);
                    }
                    o[j] = q;
                }
                store(p.da, row, s, o);
            }
            if (--left == 0 && p.slices == 0 && p.sums) leave_group(row);
        });
    }
    if (p.sums) {
        float* part = p.part + index * V * cols + col0;
        auto one = [&](int c, float a0, float a1, float b0, float b1) {
            part[c] = a0;
            if (p.slices > 0) part[cols + c] = a1;
            if constexpr (LAYER) {
                part[2 * cols + c] = b0;
                if (p.slices > 0) part[3 * cols + c] = b1;
            }
        };
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int k = s * P + j, l = LAYER ? k : 0;
                const float2 b0 = LAYER ? sum1[l] : both(0.0f), b1 = LAYER ? sumB[l] : both(0.0f);
                if (in(s, 2 * j)) one(column(s, 2 * j), sum0[k].x, sumA[k].x, b0.x, b1.x);
                if (in(s, 2 * j + 1)) one(column(s, 2 * j + 1), sum0[k].y, sumA[k].y, b0.y, b1.y);
            }
    }
    if constexpr (CLUSTER) cg::this_cluster().sync();  // no CTA leaves while another may still write to it
}

// ---- host side -------------------------------------------------------------

// The layout of a pass over `tensors` matrices, or warps = 0 when a row does not fit: 8 columns
// a thread at most, the fewest CTAs a row that this allows with three stages of ring (four where they
// fit), and several teams in a CTA for short rows.
template <class T>
BwShape bwd_shape(int cols, int tensors, bool odd, int* slots) {
    constexpr int E = 16 / static_cast<int>(sizeof(T));
    constexpr int kMaxSlots = 8 / E;
    constexpr int kLimit = 226 * 1024;
    BwShape g = {};
    const int vecs = (cols + E - 1) / E;
    for (g.cluster = 1; g.cluster <= kBwMaxCluster; g.cluster *= 2) {
        g.cta_vecs = (vecs + g.cluster - 1) / g.cluster;
        const int s = (g.cta_vecs + 32 * kBwMaxWarps - 1) / (32 * kBwMaxWarps);
        if (s > kMaxSlots) continue;
        *slots = s;
        g.warps = (g.cta_vecs + 32 * s - 1) / (32 * s);
        g.teams = g.cluster > 1 ? 1 : std::max(1, 8 / g.warps);
        g.tensors = tensors;
        g.tensor_bytes = g.cta_vecs * 16 + (odd ? 16 : 0);
        const int stage = g.teams * tensors * g.tensor_bytes;
        const int fixed = bwd_fixed_bytes(g);
        for (g.stages = kBwMaxStages; g.stages >= 3; --g.stages)
            if (fixed + g.stages * stage <= kLimit) return g;
    }
    g.warps = 0;
    return g;
}

template <class T, bool LAYER, int S, bool ODD, bool CLUSTER, int MODE, int THREADS, int CTAS>
cudaError_t bwd_go(const BlockBwArgs& in, const BwShape& g, cudaStream_t stream) {
    BlockBwArgs a = in;
    const int threads = g.teams * g.warps * 32;
    const size_t smem = bwd_fixed_bytes(g) + static_cast<size_t>(g.teams) * g.stages * g.tensors * g.tensor_bytes;
    const auto kernel = bwd_kernel<T, LAYER, S, ODD, CLUSTER, MODE, THREADS, CTAS>;
    const int64_t ctas = resident_ctas(reinterpret_cast<const void*>(kernel), threads, smem, g.cluster);
    if (ctas < 1) return cudaErrorInvalidConfiguration;
    block_slabs(&a, std::min(ctas * g.teams / g.cluster, block_slab_limit(a.rows, a.cols)));
    const unsigned grid = static_cast<unsigned>((a.slabs + g.teams - 1) / g.teams * g.cluster);
    cudaError_t e = launch_dependent(kernel, dim3(grid), threads, smem, g.cluster, stream, a, g);
    if (e != cudaSuccess || !a.sums) return e;
    return launch_block_finish(LAYER ? TR_NORM_LAYER : TR_NORM_RMS, a, stream);
}

// Aligned rows of one CTA are compiled for each pair of norms, and for CTAs of at most 320 threads
// with registers for two an SM.
template <class T, bool LAYER, int S, int MODE>
cudaError_t bwd_aligned(const BlockBwArgs& a, const BwShape& g, cudaStream_t stream) {
    if constexpr (S == 1) {
        if (g.teams * g.warps <= 10) return bwd_go<T, LAYER, S, false, false, MODE, 320, 2>(a, g, stream);
    }
    return bwd_go<T, LAYER, S, false, false, MODE, 512, 1>(a, g, stream);
}

template <class T, bool LAYER, int S>
cudaError_t bwd_slots(bool odd, const BlockBwArgs& a, const BwShape& g, cudaStream_t stream) {
    if (g.cluster > 1)
        return odd ? bwd_go<T, LAYER, S, true, true, 0, 512, 1>(a, g, stream) : bwd_go<T, LAYER, S, false, true, 0, 512, 1>(a, g, stream);
    if (odd) return bwd_go<T, LAYER, S, true, false, 0, 512, 1>(a, g, stream);
    if (a.pre && a.post) return bwd_aligned<T, LAYER, S, TR_BLOCK_PRE | TR_BLOCK_POST>(a, g, stream);
    return a.pre ? bwd_aligned<T, LAYER, S, TR_BLOCK_PRE>(a, g, stream) : bwd_aligned<T, LAYER, S, TR_BLOCK_POST>(a, g, stream);
}

template <class T, bool LAYER>
cudaError_t bwd_kind(const BlockBwArgs& a, bool* done, cudaStream_t stream) {
    const int tensors = (a.pre ? 2 : 0) + (a.post || a.dgate ? 1 : 0) + (a.dh ? 1 : 0);
    const void* read[4] = {a.pre ? a.h : nullptr, a.pre ? a.dy : nullptr, a.post || a.dgate ? a.a : nullptr, a.dh};
    const void* written[2] = {a.dx, a.da};
    bool odd = a.cols % (16 / static_cast<int>(sizeof(T))) != 0;
    for (const void* m : read) odd |= reinterpret_cast<uintptr_t>(m) % 16 != 0;
    for (const void* m : written) odd |= reinterpret_cast<uintptr_t>(m) % 16 != 0;
    int slots = 0;
    const BwShape g = bwd_shape<T>(a.cols, tensors, odd, &slots);
    *done = g.warps > 0;
    if (!*done) return cudaSuccess;
    if constexpr (sizeof(T) == 4) {
        if (slots == 2) return bwd_slots<T, LAYER, 2>(odd, a, g, stream);
    }
    return bwd_slots<T, LAYER, 1>(odd, a, g, stream);
}

}  // namespace block
}  // namespace tr
