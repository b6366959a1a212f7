// A team of warps on the rows of a slab: the pieces that both directions of the block norms share.
//
// A thread owns the same 4 to 16 columns of every row. Rows come through a ring of shared-memory
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
#include <cmath>
#include <initializer_list>

#include "tr_block.cuh"
#include "tr_block.h"
#include "tr_internal.h"
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
    int params;        // bytes of parameters a thread keeps in shared memory (0: in its registers)
    int sampled;       // bytes of a stage that each warp keeps for itself (LayerNorm's shifts; see RowStart)
};

// Shared memory of a team's exchanges (up to eight values: two halves of 8 floats for each warp of a row, after two
// mbarriers) and row starts; of all teams; and of the whole CTA.
__host__ __device__ inline int exchange_bytes(const RowShape& g) { return 16 + 2 * 8 * 4 * g.warps * g.cluster; }
__host__ __device__ inline int team_bytes(const RowShape& g) {
    return exchange_bytes(g) + g.warps * (g.stages * g.sampled + 32 * g.params);
}
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

// One team's exchange: N (2, 4 or 8) sums over all warps of a row.
//
// In a cluster every warp sends its sums to all CTAs with asynchronous stores that count bytes on the
// receiver's mbarrier, so a warp waits for the sums alone. (A cluster barrier instead has to order the
// warps' output stores as well: 1.9 k cycles a row more at 8192 x 8192 bf16, 232 us.)
template <bool CLUSTER, int N>
struct Exchange {
    static constexpr int kLanes = 32 / N;  // lanes of a warp that end with the same value
    int entries;     // warps of the row
    int team, warps;
    uint32_t put;    // where this lane's value goes, in the half of this CTA's 2 x N x entries floats that is next
    uint32_t take;   // and where it reads from
    int flip;        // to the other half
    uint64_t* bars;  // a cluster's: one mbarrier a half
    unsigned* err;
    int buf = 0;
    unsigned phase = 0;  // of both mbarriers, one bit each
    // After a wait that gave up all sums of the warp are NaN, so what is computed from them is no number, and the
    // kernel's end sets the error word. (Leaving the stores out instead takes a test at each: backward 8192 x 8192 bf16
    // 190 us against 174.) Later waits of the kernel are short then. The CTAs' phases may be out of step, so that a store to
    // a CTA is not waited for: a warp that gave up keeps its CTA for a while after the last barrier, until all have come in.
    static constexpr unsigned kLimitNs = 2000000000u, kLateNs = 1000000u;
    float start;  // of the sums over the warps: 0, or NaN

    // `entry`: this warp's place among the row's. Addresses are found once: the exchange is a fifth of the instructions.
    // `first`: 0, or (testing) NaN, as if a wait had given up before.
    __device__ __forceinline__ Exchange(char* smem, int entries_, int entry, int team_, int warps_, unsigned* err_, float first)
        : entries(entries_), team(team_), warps(warps_), bars(reinterpret_cast<uint64_t*>(smem)), err(err_), start(first) {
        const int lane = threadIdx.x & 31;
        const uint32_t slot = smem_addr(smem + 16);
        put = slot + 4 * (entry * N + lane / kLanes);
        take = slot + 4 * ((lane & 15) * N + (lane >> 4) * (N / 2));
        flip = 4 * N * entries;
    }

    static __device__ __forceinline__ void spread(float r, float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(kFull, r, kLanes * i);
    }
    // Before the first exchange (and the cluster's start barrier): one arrival a phase, by the CTA's first thread.
    __device__ __forceinline__ void init() {
        if constexpr (CLUSTER) {
            if (threadIdx.x == 0) {
                mbar_init(bars, 1);
                mbar_init(bars + 1, 1);
                fence_barrier_init();
            }
        }
    }
    // After the last exchange: waits that gave up are reported, and no CTA of the cluster leaves while another may still write
    // to it. (testing, `debug`: one more wait, on a phase that nothing completes)
    __device__ __forceinline__ void finish(int debug) {
        if constexpr (CLUSTER) {
            if ((debug & kDebugForceTimeout) && threadIdx.x == 0) mbar_wait_bounded(bars + buf, (phase >> buf) & 1, kLateNs, err);
            if (start != 0.0f) atomicOr(err, kErrWaitTimeout);
            cg::this_cluster().sync();
            if (start != 0.0f)
                for (const unsigned long long t0 = global_ns(); global_ns() - t0 < kLateNs;) __nanosleep(1000);
        }
    }

    // v summed over the row
    __device__ __forceinline__ void sums(float (&v)[N]) {
        const int lane = threadIdx.x & 31;
        const float r = halving_sums<N, 16>(v, lane);  // value i in lanes kLanes i ..
        if (!CLUSTER && entries == 1) return spread(r, v);
        // (this half is free: a warp comes here after the last exchange, which had every warp's sums, and a
        // warp sends those after it has read the half before)
        if constexpr (CLUSTER) {
            const int ctas = static_cast<int>(cg::this_cluster().num_blocks());
            uint64_t* bar = bars + buf;
            if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(entries * N * 4));
            for (int c = lane % kLanes; c < ctas; c += kLanes) {  // the lanes of a value take the CTAs in turn
                uint32_t to, signal;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(put), "r"(c));
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(signal) : "r"(smem_addr(bar)), "r"(c));
                asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(to),
                             "r"(__float_as_uint(r)), "r"(signal)
                             : "memory");
            }
            if (!wait(bar, (phase >> buf) & 1, start == 0.0f ? kLimitNs : kLateNs)) start = NAN;
            phase ^= 1u << buf;
            buf ^= 1;
        } else {
            if (lane % kLanes == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(put), "f"(r) : "memory");
            team_barrier(team, warps);
        }
        // 16 entries at a time, half the values a lane
        float t[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) t[i] = CLUSTER ? start : 0.0f;
        auto add = [&](uint32_t from) {
            if constexpr (N == 8) {
                float f[4];
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
                             : "r"(from)
                             : "memory");
#pragma unroll
                for (int i = 0; i < N / 2; ++i) t[i] += f[i];
            } else if constexpr (N == 4) {
                float f[2];
                asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(f[0]), "=f"(f[1]) : "r"(from) : "memory");
                t[0] += f[0];
                t[N / 2 - 1] += f[1];
            } else {
                float f;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(from) : "memory");
                t[0] += f;
            }
        };
        if constexpr (CLUSTER) {
            for (int e = lane & 15, i = 0; e < entries; e += 16, ++i) add(take + i * 64 * N);
        } else {
            if ((lane & 15) < entries) add(take);
        }
        put += flip;
        take += flip;
        flip = -flip;
        spread(halving_sums<N / 2, 8>(t, lane), v);
    }

private:
    static __device__ __forceinline__ bool wait(uint64_t* bar, unsigned parity, unsigned limit_ns) {
        auto done = [&]() {
            uint32_t ok;
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(ok)
                : "r"(smem_addr(bar)), "r"(parity)
                : "memory");
            return ok != 0;
        };
        if (done()) return true;
        const unsigned long long t0 = global_ns();
        while (global_ns() - t0 < limit_ns)
            if (done()) return true;
        return false;
    }
};

// How a row lies over the threads: aligned with all slots of all threads in the row (no test is left in the
// inner loops, which are short of issue slots), aligned, or in the odd layout.
enum Layout : int { LAYOUT_FULL, LAYOUT_ALIGNED, LAYOUT_ODD };

// Where a warp finds a row's first 32 elements. Loading them from memory when they are needed would wait for
// its full queues (twice the time of the whole kernel), so:
// * aligned rows: every warp copies them for itself, with the row (another warp's copy could only be read
//   after a barrier);
// * other rows in one CTA: in the ring, after the barrier that the layout has anyway;
// * other rows of a cluster: in memory all the same.
constexpr int kRowStartBytes = 128;
template <class T, int LAYOUT, bool CLUSTER>
struct RowStart {
    static constexpr bool OWN = LAYOUT != LAYOUT_ODD;
    int64_t row_bytes;
    int at;       // this lane's 16 bytes of a copy
    int c;        // and its column (rows shorter than 32 are gone over again)
    bool copies;  // whether the row has those 16 bytes

    __device__ __forceinline__ RowStart(int cols, int64_t row_bytes_) : row_bytes(row_bytes_) {
        const int lane = static_cast<int>(threadIdx.x & 31);
        at = lane * 16;
        c = cols < 32 ? lane % cols : lane;
        copies = at < static_cast<int>(min(static_cast<int64_t>(32 * sizeof(T)), row_bytes));
    }
    __device__ __forceinline__ void fetch(const void* matrix, int64_t row, char* to) const {
        if constexpr (OWN) {
            if (copies) cp_async16(smem_addr(to) + at, static_cast<const char*>(matrix) + (row * row_bytes + at));
        }
    }
    // This lane's element: own: the warp's copy, after the row's copies and __syncwarp(); staged: the row in the ring.
    __device__ __forceinline__ float get(const void* matrix, int64_t row, const char* own, const char* staged) const {
        if constexpr (OWN) return to_float(reinterpret_cast<const T*>(own)[c]);
        const char* start = static_cast<const char*>(matrix) + row * row_bytes;
        if constexpr (CLUSTER) return to_float(reinterpret_cast<const T*>(start)[c]);
        return to_float(reinterpret_cast<const T*>(staged + (reinterpret_cast<uintptr_t>(start) & 15))[c]);
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

// A thread's share of a row. `mine` columns of the row, from byte `base` on, belong to this CTA.
template <class T, int S, int LAYOUT>
struct Lanes {
    static constexpr bool ODD = LAYOUT == LAYOUT_ODD, FULL = LAYOUT == LAYOUT_FULL;
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
    __device__ __forceinline__ bool in(int s, int e) const { return FULL || (ODD ? column(s, e) < mine : t + tt * s < vecs); }
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
                if (FULL || k < vecs) cp_async16(smem_addr(to) + k * 16, from + k * 16);
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
            if (FULL || t + tt * s < vecs) q = *reinterpret_cast<const uint4*>(m + (t + tt * s) * 16);
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
            if (FULL || t + tt * s < vecs) {
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
    // floats of slot s's columns to a vector (from this CTA's first column on): 16 bytes at a time where the
    // layout allows it (a thread's columns are adjacent, so single floats would go 32 sectors to a store)
    __device__ __forceinline__ void put_floats(float* o, int s, const float2 (&v)[P]) const {
        if (!ODD && aligned16(o)) {
            if (FULL || t + tt * s < vecs)
#pragma unroll
                for (int j = 0; j < P; j += 2)
                    *reinterpret_cast<float4*>(o + column(s, 2 * j)) = make_float4(v[j].x, v[j].y, v[j + 1].x, v[j + 1].y);
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                if (in(s, 2 * j)) o[column(s, 2 * j)] = v[j].x;
                if (in(s, 2 * j + 1)) o[column(s, 2 * j + 1)] = v[j].y;
            }
        }
    }
    __device__ __forceinline__ void get_floats(const float* o, int s, float2 (&v)[P]) const {
        if (!ODD && aligned16(o)) {
            if (FULL || t + tt * s < vecs)
#pragma unroll
                for (int j = 0; j < P; j += 2) {
                    const float4 q = *reinterpret_cast<const float4*>(o + column(s, 2 * j));
                    v[j] = make_float2(q.x, q.y);
                    v[j + 1] = make_float2(q.z, q.w);
                }
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                if (in(s, 2 * j)) v[j].x = o[column(s, 2 * j)];
                if (in(s, 2 * j + 1)) v[j].y = o[column(s, 2 * j + 1)];
            }
        }
    }
    // a parameter vector (from this CTA's first column on) at slot s's columns
    __device__ __forceinline__ void param(const float* w, int s, float absent, float2 (&v)[P]) const {
#pragma unroll
        for (int j = 0; j < P; ++j) v[j] = both(absent);
        if (!w) return;
        if (!ODD && aligned16(w)) {
            if (FULL || t + tt * s < vecs)
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

// The layout of a pass over `tensors` matrices, or warps = 0 when a row does not fit: at most `most` (8 or 16)
// columns a thread, the fewest CTAs a row that this allows with a ring of three stages (`stages` where they
// fit), and several teams in a CTA for short rows. 16-bit rows of 1024 columns and more take
// 16 a thread where that is allowed: half the warps to an exchange, two CTAs of 256 threads an SM at 4096 columns
// (forward, 16384 x 4096 bf16: LayerNorm 89 us, RMSNorm 83; with 8 a thread 123 and 83).
template <class T>
RowShape row_shape(int cols, int tensors, bool odd, bool layer, int stages, int params, int most, int* slots) {
    constexpr int E = 16 / static_cast<int>(sizeof(T));
    const int kMaxSlots = most / E;
    constexpr int kLimit = 226 * 1024;
    RowShape g = {};
    const int vecs = (cols + E - 1) / E;
    for (g.cluster = 1; g.cluster <= kMaxCluster; g.cluster *= 2) {
        g.cta_vecs = (vecs + g.cluster - 1) / g.cluster;
        int s = (g.cta_vecs + 32 * kMaxWarps - 1) / (32 * kMaxWarps);
        if (s > kMaxSlots) continue;
        if (most == 16 && sizeof(T) == 2 && g.cta_vecs >= 128) s = 2;
        *slots = s;
        g.warps = (g.cta_vecs + 32 * s - 1) / (32 * s);
        g.teams = g.cluster > 1 ? 1 : std::max(1, 8 / g.warps);
        g.tensors = tensors;
        g.tensor_bytes = g.cta_vecs * 16 + (odd ? 16 : 0);
        g.sampled = layer && !odd ? 2 * kRowStartBytes : 0;
        g.params = g.cluster == 1 ? params : 0;
        for (g.stages = stages; g.stages >= 3; --g.stages)
            if (row_smem(g) <= kLimit) return g;
    }
    g.warps = 0;
    return g;
}

// Most columns a thread of each direction, and whether rows of `slots` slots a thread are ever split over a cluster: a row
// goes to twice as many CTAs only where its slots in half as many would be more than `most` columns.
constexpr int kFwdColumns = 16, kBwdColumns = 8;
template <class T>
constexpr bool cluster_slots(int slots, int most) {
    return slots > most / 2 / (16 / static_cast<int>(sizeof(T)));
}

// Whether all of a row's slots are in the row: every CTA has the same, and a team's threads all have theirs.
template <class T>
bool row_full(const RowShape& g, int cols, int slots) {
    return g.cta_vecs == g.warps * 32 * slots && static_cast<int64_t>(g.cta_vecs) * g.cluster * (16 / static_cast<int>(sizeof(T))) == cols;
}

// Whether every row of these matrices starts and ends on 16 bytes.
inline bool rows_aligned(int64_t row_bytes, std::initializer_list<const void*> matrices) {
    bool ok = row_bytes % 16 == 0;
    for (const void* m : matrices) ok = ok && reinterpret_cast<uintptr_t>(m) % 16 == 0;
    return ok;
}

}  // namespace block
}  // namespace tr
