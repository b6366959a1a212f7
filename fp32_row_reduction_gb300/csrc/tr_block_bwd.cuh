// The gated residual norm's backward with the rows on chip (see k_block_bwd.cu for
// the formulas).
//
// HBM-bound: h, a, dy and dh are read and dx and da written once. A team of W warps
// takes a row at a time, thread t owning the same S x E columns (E elements are 16 bytes) of
// every row of its slab, so the column sums stay in its registers until the slab
// ends. Rows come through a ring of shared-memory stages filled by cp.async while the row
// before is worked on. The row sums need two exchanges between the team's warps
// (LayerNorm three: means first, then everything about them).
//
// Two layouts of a row over the threads:
// * aligned rows (every row of every matrix starts on 16 bytes): slot s of thread t is the
//   16 bytes s x team + t; a thread reads back what it copied itself, so no barrier;
// * other rows: the 16-byte granules that cover the row are copied as they lie, the
//   team meets at a barrier, and element k of thread t is column k x team + t, which any phase
//   reads without bank conflicts.
#pragma once

#include <algorithm>

#include "tr_block.cuh"
#include "tr_block.h"
#include "tr_launch.h"

namespace tr {
namespace block {

constexpr int kBwMaxWarps = 16;
constexpr int kBwMaxStages = 4;
constexpr int kBwMaxSums = 3;  // row sums of one exchange

// How a launch maps rows onto threads and shared memory.
struct BwShape {
    int warps;         // a team's
    int teams;         // of a CTA
    int stages;        // of a team's ring
    int tensors;       // matrices read: h and dy (pre), a, dh, in this order
    int tensor_bytes;  // shared memory of one matrix's row
};

// Shared memory of the teams' exchanges.
__host__ __device__ inline int bwd_fixed_bytes(const BwShape& g) { return g.teams * 2 * kBwMaxSums * kBwMaxWarps * 4; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// At most `n` groups of this thread still in flight.
__device__ __forceinline__ void cp_async_wait_n(int n) {
    switch (n) {
        case 0: cp_async_wait<0>(); break;
        case 1: cp_async_wait<1>(); break;
        case 2: cp_async_wait<2>(); break;
        default: cp_async_wait<3>(); break;
    }
}

// A barrier of one team's threads (a team of one warp needs no more than the warp's own).
__device__ __forceinline__ void team_barrier(int team, int warps) {
    if (warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(warps * 32) : "memory");
}

// N sums over a team's threads. `slot` holds 2 x kBwMaxSums x kBwMaxWarps floats of the team; the
// halves alternate, so consecutive sums need one barrier each.
template <int N>
__device__ __forceinline__ void team_sums(float (&v)[N], float* slot, int& buf, int team, int warps) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kFull, v[i], o);
    if (warps == 1) return;
    float* s = slot + buf * kBwMaxSums * kBwMaxWarps;
    buf ^= 1;
    const int lane = threadIdx.x & 31;
    const int w = static_cast<int>(threadIdx.x >> 5) - team * warps;
    if (lane < N) {  // lane i stores sum i
        float mine = v[0];
#pragma unroll
        for (int i = 1; i < N; ++i) mine = lane == i ? v[i] : mine;
        s[lane * kBwMaxWarps + w] = mine;
    }
    team_barrier(team, warps);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float t = 0.0f;
        for (int j = 0; j < warps; j += 4) {  // slots past the team's warps hold zero
            const float4 q = *reinterpret_cast<const float4*>(s + i * kBwMaxWarps + j);
            t += (q.x + q.y) + (q.z + q.w);
        }
        v[i] = t;
    }
}

template <class T, bool LAYER, int S, bool ODD>
__global__ void __launch_bounds__(32 * kBwMaxWarps)
    bwd_kernel(const BlockBwArgs p, const BwShape g) {
    constexpr int E = 16 / static_cast<int>(sizeof(T));
    constexpr int C = S * E;       // columns of a thread
    constexpr int V = LAYER ? 4 : 2;
    constexpr int N1 = kBwMaxSums, N3 = LAYER ? 2 : 1;
    // the parameters of a thread's columns stay in registers where the column sums leave room
    constexpr bool PREG = LAYER ? C <= 8 : C <= 16;
    extern __shared__ uint4 smem[];
    const int team_threads = g.warps * 32;
    const int team = static_cast<int>(threadIdx.x) / team_threads;
    const int t = static_cast<int>(threadIdx.x) - team * team_threads;
    const int cols = p.cols;
    const float inv_n = 1.0f / static_cast<float>(cols);
    float* slot = reinterpret_cast<float*>(smem) + team * (2 * N1 * kBwMaxWarps);
    for (int i = t; i < 2 * N1 * kBwMaxWarps; i += team_threads) slot[i] = 0.0f;
    int buf = 0;
    const int stage_bytes = g.tensors * g.tensor_bytes;
    char* ring = reinterpret_cast<char*>(smem) + bwd_fixed_bytes(g) + team * g.stages * stage_bytes;
    team_barrier(team, g.warps);
    pdl_enter();

    auto column = [&](int s, int e) { return ODD ? t + team_threads * (s * E + e) : (t + team_threads * s) * E + e; };
    const int vecs = cols / E;  // aligned rows: 16-byte slots of a row

    const int64_t index = static_cast<int64_t>(blockIdx.x) * g.teams + team;
    if (index >= p.slabs) return;
    const SlabRows slab = slab_rows(p, index);
    // ---- the ring: h and dy (pre), a, dh, each where there is one ----
    const bool need_a = p.post || p.dgate;
    const int at_dy = p.pre ? g.tensor_bytes : 0;
    const int at_a = p.pre ? 2 * g.tensor_bytes : 0;
    const int at_dh = at_a + (need_a ? g.tensor_bytes : 0);
    const int64_t row_bytes = static_cast<int64_t>(cols) * static_cast<int>(sizeof(T));
    auto fetch_one = [&](const void* matrix, int64_t row, char* to) {
        const char* from = static_cast<const char*>(matrix) + row * row_bytes;
        if constexpr (!ODD) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int k = t + team_threads * s;
                if (k < vecs) cp_async16(smem_addr(to) + k * 16, from + k * 16);
            }
        } else {
            const int phase = static_cast<int>(reinterpret_cast<uintptr_t>(from) & 15);
            const int granules = (phase + static_cast<int>(row_bytes) + 15) >> 4;
            const char* lo = static_cast<const char*>(matrix);
            const char* hi = lo + p.rows * row_bytes;
            for (int k = t; k < granules; k += team_threads) {
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
            if (p.pre) {
                fetch_one(p.h, row, to);
                fetch_one(p.dy, row, to + at_dy);
            }
            if (need_a) fetch_one(p.a, row, to + at_a);
            if (p.dh) fetch_one(p.dh, row, to + at_dh);
        }
        cp_async_commit();
    };
    // E columns of slot s of the matrix at `m` (whose row starts `phase` bytes in); 0 outside the row
    auto load = [&](const char* m, int phase, int s, float (&v)[E]) {
        if constexpr (!ODD) {
            if (t + team_threads * s < vecs) {
                const uint4 q = *reinterpret_cast<const uint4*>(m + (t + team_threads * s) * 16);
                const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
                for (int i = 0; i < E; ++i) v[i] = to_float(e[i]);
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i) v[i] = 0.0f;
            }
        } else {
            const T* e = reinterpret_cast<const T*>(m + phase);
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = column(s, i) < cols ? to_float(e[column(s, i)]) : 0.0f;
        }
    };
    auto store = [&](void* out, int64_t row, int s, const float (&v)[E]) {
        if constexpr (!ODD) {
            const int k = t + team_threads * s;
            if (k < vecs) {
                uint4 q;
                T* e = reinterpret_cast<T*>(&q);
#pragma unroll
                for (int i = 0; i < E; ++i) e[i] = from_float<T>(v[i]);
                *reinterpret_cast<uint4*>(static_cast<char*>(out) + row * row_bytes + k * 16) = q;
            }
        } else {
            T* o = static_cast<T*>(out) + row * cols;
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (column(s, i) < cols) o[column(s, i)] = from_float<T>(v[i]);
        }
    };
    // E floats of a parameter vector at slot s's columns
    auto param = [&](const float* w, int s, float absent, float (&v)[E]) {
        if (!ODD && w && aligned16(w)) {
#pragma unroll
            for (int i = 0; i < E; i += 4) {
                float4 q = make_float4(absent, absent, absent, absent);
                if (t + team_threads * s < vecs) q = ld_param4(w + column(s, i));
                v[i] = q.x;
                v[i + 1] = q.y;
                v[i + 2] = q.z;
                v[i + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = w && column(s, i) < cols ? __ldg(w + column(s, i)) : absent;
        }
    };

    // the slab's column sums dy hh and dy; those of the running gate row, D ah and D
    float sum0[C] = {}, sumA[C] = {};
    float sum1[LAYER ? C : 1] = {}, sumB[LAYER ? C : 1] = {};

    float w_reg[PREG ? C : 1], q_reg[PREG ? C : 1];  // w;  bs gate w_post
    const float* gate_row = nullptr;
    auto load_w = [&](int s, float (&v)[E]) { param(p.pre ? p.pre_w : nullptr, s, 1.0f, v); };
    auto load_q = [&](int s, float (&v)[E]) {
        float o[E];
        param(p.post ? p.post_w : nullptr, s, 1.0f, o);
        param(gate_row, s, 1.0f, v);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] *= p.bs * o[i];
    };
    auto get_w = [&](int s, float (&v)[E]) {
        if constexpr (PREG) {
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = w_reg[s * E + i];
        } else {
            load_w(s, v);
        }
    };
    auto get_q = [&](int s, float (&v)[E]) {
        if constexpr (PREG) {
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = q_reg[s * E + i];
        } else {
            load_q(s, v);
        }
    };
    auto enter_group = [&](int64_t row) {
        gate_row = p.gate ? p.gate + row / p.group_rows * cols : nullptr;
        if constexpr (PREG) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float v[E];
                load_q(s, v);
#pragma unroll
                for (int i = 0; i < E; ++i) q_reg[s * E + i] = v[i];
            }
        }
    };
    if constexpr (PREG) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float v[E];
            load_w(s, v);
#pragma unroll
            for (int i = 0; i < E; ++i) w_reg[s * E + i] = v[i];
        }
    }

    // a whole group is done: its gate gradient is final, and its share of the post-norm's column
    // sums goes to the slab's partials, which no other thread touches
    float* const part = p.part + index * V * cols;
    bool flushed = false;
    auto leave_group = [&](int64_t row) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float o[E], ob[E], gate[E];
            param(p.post ? p.post_w : nullptr, s, 1.0f, o);
            param(p.post ? p.post_b : nullptr, s, 0.0f, ob);
            param(gate_row, s, 1.0f, gate);
            float* dg = p.dgate ? p.dgate + row / p.group_rows * cols : nullptr;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = column(s, i), k = s * E + i;
                if (c >= cols) continue;
                if (dg) dg[c] = p.bs * (LAYER ? fmaf(o[i], sumA[k], ob[i] * sumB[LAYER ? k : 0]) : o[i] * sumA[k]);
                part[cols + c] = fmaf(gate[i], sumA[k], flushed ? part[cols + c] : 0.0f);
                sumA[k] = 0.0f;
                if constexpr (LAYER) {
                    part[3 * cols + c] = fmaf(gate[i], sumB[k], flushed ? part[3 * cols + c] : 0.0f);
                    sumB[k] = 0.0f;
                }
            }
        }
        flushed = true;
    };

    for (int i = 0; i + 1 < g.stages; ++i) fetch(slab.begin + i, i);
    int stage = 0, fill = g.stages - 1;
    int64_t left = 0;  // rows of the running group still to come
    for (int64_t row = slab.begin; row < slab.end; ++row) {
        if (left == 0) {
            enter_group(row);
            left = p.slices > 0 ? slab.end - slab.begin : p.group_rows;
        }
        cp_async_wait_n(g.stages - 2);
        if constexpr (ODD) team_barrier(team, g.warps);
        // (every thread of the team is done with the row before: the exchanges below follow its last
        // reads in the odd layout, and an aligned row's slots are the thread's own)
        fetch(row + g.stages - 1, fill);
        fill = fill + 1 == g.stages ? 0 : fill + 1;
        const char* m = ring + stage * stage_bytes;
        stage = stage + 1 == g.stages ? 0 : stage + 1;
        const char *mh = m, *mdy = m + at_dy, *ma = m + at_a, *mdh = m + at_dh;
        const int64_t off = row * row_bytes;
        auto phase_of = [&](const void* base) {
            return ODD ? static_cast<int>((reinterpret_cast<uintptr_t>(base) + off) & 15) : 0;
        };
        const int fh = phase_of(p.h), fdy = phase_of(p.dy), fa = phase_of(p.a), fdh = phase_of(p.dh);

        float mean_h = 0.0f, mean_a = 0.0f, c1 = 0.0f;
        if constexpr (LAYER) {
            float v[N1] = {0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float x[E], y[E], w[E];
                if (p.pre) {
                    load(mh, fh, s, x);
                    load(mdy, fdy, s, y);
                    get_w(s, w);
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        v[0] += x[i];
                        v[2] = fmaf(y[i], w[i], v[2]);
                    }
                }
                if (p.post) {
                    load(ma, fa, s, x);
#pragma unroll
                    for (int i = 0; i < E; ++i) v[1] += x[i];
                }
            }
            team_sums<N1>(v, slot, buf, team, g.warps);
            mean_h = v[0] * inv_n;
            mean_a = v[1] * inv_n;
            c1 = v[2] * inv_n;
        }
        float rh = 0.0f, ra = 0.0f, k2 = 0.0f;  // k2 = r_h^2 mean(u (h - mean)): D = dh + r_h (u - c1 - (h - mean) k2)
        {
            float v[N1] = {0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float x[E], y[E], w[E];
                if (p.pre) {
                    load(mh, fh, s, x);
                    load(mdy, fdy, s, y);
                    get_w(s, w);
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const float c = LAYER && column(s, i) < cols ? x[i] - mean_h : x[i];
                        v[0] = fmaf(c, c, v[0]);
                        v[2] = fmaf(y[i] * w[i], c, v[2]);
                    }
                }
                if (p.post) {
                    load(ma, fa, s, x);
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const float c = LAYER && column(s, i) < cols ? x[i] - mean_a : x[i];
                        v[1] = fmaf(c, c, v[1]);
                    }
                }
            }
            team_sums<N1>(v, slot, buf, team, g.warps);
            if (p.pre) {
                rh = 1.0f / sqrtf(v[0] * inv_n + p.eps);
                k2 = v[2] * inv_n * rh * rh;
            }
            if (p.post) ra = 1.0f / sqrtf(v[1] * inv_n + p.eps);
        }
        // D, the column sums, dx, and the sums of q and q ah
        float d[C];
        float v[N3] = {};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float x[E], y[E], w[E], o[E];
            if (p.dh) {
                load(mdh, fdh, s, o);
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i) o[i] = 0.0f;
            }
            if (p.pre) {
                load(mh, fh, s, x);
                load(mdy, fdy, s, y);
                get_w(s, w);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float c = x[i] - mean_h;
                    sum0[s * E + i] = fmaf(y[i] * rh, c, sum0[s * E + i]);
                    if (LAYER) sum1[LAYER ? s * E + i : 0] += y[i];
                    const float u = fmaf(y[i], w[i], -c1);
                    o[i] = fmaf(rh, fmaf(-c, k2, u), o[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < E; ++i) {
                d[s * E + i] = o[i];
                o[i] *= p.rs;
            }
            store(p.dx, row, s, o);
            if (need_a) {
                load(ma, fa, s, x);
                if (p.post) {
                    get_q(s, w);
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const float c = LAYER && column(s, i) < cols ? x[i] - mean_a : x[i];
                        const float q = d[s * E + i] * w[i];
                        v[0] = fmaf(q, c, v[0]);
                        if (LAYER && column(s, i) < cols) v[N3 - 1] += q;
                    }
                }
            }
        }
        if (p.post) team_sums<N3>(v, slot, buf, team, g.warps);
        const float e1 = LAYER ? v[N3 - 1] * inv_n : 0.0f;
        const float e2 = v[0] * inv_n * ra * ra;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float x[E], w[E], o[E];
            get_q(s, w);
            if (need_a) load(ma, fa, s, x);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int k = s * E + i;
                float q = d[k] * w[i];
                if (need_a) {
                    float ah = x[i];
                    if (p.post) {
                        const float c = x[i] - mean_a;
                        q = ra * (fmaf(-c, e2, q) - e1);
                        ah = c * ra;
                    }
                    sumA[k] = fmaf(d[k], ah, sumA[k]);
                    if (LAYER) sumB[LAYER ? k : 0] += d[k];
                }
                o[i] = q;
            }
            store(p.da, row, s, o);
        }
        if (--left == 0 && p.slices == 0 && p.sums) leave_group(row);
    }
    if (!p.sums) return;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = column(s, i), k = s * E + i;
            if (c >= cols) continue;
            part[c] = sum0[k];
            if (p.slices > 0) part[cols + c] = sumA[k];
            if constexpr (LAYER) {
                part[2 * cols + c] = sum1[k];
                if (p.slices > 0) part[3 * cols + c] = sumB[k];
            }
        }
}

// ---- host side -------------------------------------------------------------

// The layout of a pass over `tensors` matrices, or warps = 0 when the row does not fit:
// as few slots a thread as 16 warps allow, the warps the row needs, several teams in a CTA for short
// rows, and as many stages (2 .. 4) as leave two CTAs an SM, or one.
template <class T, bool LAYER>
BwShape bwd_shape(int cols, int tensors, bool odd, int* slots) {
    constexpr int E = 16 / static_cast<int>(sizeof(T));
    BwShape g = {};
    const int vecs = (cols + E - 1) / E;
    const int s = (vecs + 32 * kBwMaxWarps - 1) / (32 * kBwMaxWarps);
    if (s > 4 || s * E > (LAYER ? 16 : 32)) return g;
    *slots = s;
    g.warps = (vecs + 32 * s - 1) / (32 * s);
    g.teams = std::max(1, 8 / g.warps);
    g.tensors = tensors;
    g.tensor_bytes = vecs * 16 + (odd ? 16 : 0);
    const int stage = g.teams * tensors * g.tensor_bytes;
    const int fixed = bwd_fixed_bytes(g);
    const int most = s * E <= 8 ? 2 : 1;  // CTAs an SM the registers allow for full teams
    for (g.stages = kBwMaxStages; g.stages > 2; --g.stages)
        if (most * (fixed + g.stages * stage + 1024) <= 227 * 1024) break;
    if (fixed + g.stages * stage > 226 * 1024) g.warps = 0;
    return g;
}

template <class T, bool LAYER, int S, bool ODD>
cudaError_t bwd_go(const BlockBwArgs& in, const BwShape& g, cudaStream_t stream) {
    BlockBwArgs a = in;
    const int threads = g.teams * g.warps * 32;
    const size_t smem = bwd_fixed_bytes(g) + static_cast<size_t>(g.teams) * g.stages * g.tensors * g.tensor_bytes;
    const auto kernel = bwd_kernel<T, LAYER, S, ODD>;
    const int64_t ctas = resident_ctas(reinterpret_cast<const void*>(kernel), threads, smem);
    if (ctas < 1) return cudaErrorInvalidConfiguration;
    block_slabs(&a, std::min(ctas * g.teams, block_slab_limit(a.rows, a.cols)));
    const unsigned grid = static_cast<unsigned>((a.slabs + g.teams - 1) / g.teams);
    cudaError_t e = launch_dependent(kernel, dim3(grid), threads, smem, stream, a, g);
    if (e != cudaSuccess || !a.sums) return e;
    return launch_block_finish(LAYER ? TR_NORM_LAYER : TR_NORM_RMS, a, stream);
}

template <class T, bool LAYER, bool ODD>
cudaError_t bwd_slots(int slots, const BlockBwArgs& a, const BwShape& g, cudaStream_t stream) {
    constexpr int E = 16 / static_cast<int>(sizeof(T));
    switch (slots) {
        case 1: return bwd_go<T, LAYER, 1, ODD>(a, g, stream);
        case 2: return bwd_go<T, LAYER, 2, ODD>(a, g, stream);
        case 3: if constexpr (3 * E <= (LAYER ? 16 : 32)) return bwd_go<T, LAYER, 3, ODD>(a, g, stream); break;
        case 4: if constexpr (4 * E <= (LAYER ? 16 : 32)) return bwd_go<T, LAYER, 4, ODD>(a, g, stream); break;
    }
    return cudaErrorInvalidValue;
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
    const BwShape g = bwd_shape<T, LAYER>(a.cols, tensors, odd, &slots);
    *done = g.warps > 0;
    if (!*done) return cudaSuccess;
    return odd ? bwd_slots<T, LAYER, true>(slots, a, g, stream) : bwd_slots<T, LAYER, false>(slots, a, g, stream);
}

}  // namespace block
}  // namespace tr
