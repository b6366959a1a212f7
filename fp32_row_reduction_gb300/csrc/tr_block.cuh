// Device pieces shared by the block norm kernels: element types and row sums.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tr_device.cuh"

namespace tr {
namespace block {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

constexpr int kReadCluster = 8;  // most CTAs of a row that is read again for each pass

// A shift for a row's LayerNorm sums: the mean of its first 32 elements, which every warp of the row finds
// alike. Sums are taken about it in one pass, and the variance is S2 / n - (S1 / n)^2; the cancellation
// costs 1 + (shift - mean)^2 / variance of precision: 1 + 1/32 for independent elements. Where it would cost more than
// 4/3 (squares_about_mean) the row's sums are taken once more, about the mean that the first ones gave.
__device__ __forceinline__ float lane_mean(float v) {
    v *= 1.0f / 32.0f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
// The sum of squares about the mean, from the sums s2 of squares and s1 about a shift that is d off the mean. `far`:
// d^2 is more than a third of the variance, and the sums are to be taken again. Otherwise a rounding u of each of a sum's
// L steps stays below (4/3 + 4/3) L u of the variance (s2 is 4/3 of it, and 2 d s1 at most as much): 70 u for the
// longest chain, 26. One row in a thousand of independent normal elements is far. All threads of a row have the same
// sums, and answer alike. What is infinite or no number stays so, and is not far.
__device__ __forceinline__ float squares_about_mean(float s2, float s1, float d, bool& far) {
    const float v = fmaf(-d, s1, s2), least = 0.75f * s2;
    far = v < least;
    return fmaxf(v, least);  // (least where v is infinity less infinity)
}
// A long sum with the rounding error of each step added up beside it (Knuth's two-sum), so that a row of 2^24 columns
// loses no more than a short one. (Totals in binary64 made the kernels twice as slow.)
struct LongSum {
    float s = 0.0f, c = 0.0f;
    __device__ __forceinline__ void add(float v) {
        const float t = s + v, w = t - s;
        c += (s - (t - w)) + (v - w);
        s = t;
    }
    __device__ __forceinline__ float value() const { return fabsf(s) <= 3.0e38f ? s + c : s; }
};

// A parameter vector that may be absent, read without a branch (loads of several columns can then be under way
// together): an absent one is a single value that every column reads.
__device__ const float g_block_values[2] = {0.0f, 1.0f};
struct ReadParam {
    const float* p;
    int step;
    __device__ __forceinline__ ReadParam(const float* w, int absent) : p(w ? w : g_block_values + absent), step(w ? 1 : 0) {}
    __device__ __forceinline__ float operator()(int c) const { return __ldg(p + static_cast<int64_t>(step) * c); }
};

// The share of a row's columns that a CTA of a cluster has, and sums over all of the row.
constexpr int kReadThreads = 1024;
constexpr int kReadSums = 6;  // most sums of one pass
template <int N>
struct Values {
    float v[N];
};
struct ReadRow {
    static constexpr int kWarps = kReadThreads / 32;
    // two halves that alternate, so consecutive sums need one barrier each
    using WarpSums = float[kReadSums][kWarps];
    using CtaSums = float[kReadSums][kReadCluster];
    int begin, end;  // columns
    WarpSums* warp;
    CtaSums* cta;
    int buf = 0;

    __device__ __forceinline__ ReadRow(int cols, WarpSums* warp_, CtaSums* cta_) : warp(warp_), cta(cta_) {
        const cg::cluster_group cl = cg::this_cluster();
        const int64_t n = cl.num_blocks(), r = cl.block_rank();
        begin = static_cast<int>(cols * r / n);
        end = static_cast<int>(cols * (r + 1) / n);
        if (n > 1) cl.sync();  // every CTA of the cluster runs before it is written to
    }
    // f(column) for this thread's columns, four loads deep: f gives what g(column, value) then takes
    template <class F, class G>
    __device__ __forceinline__ void columns(F&& f, G&& g) const {
        int c = begin + static_cast<int>(threadIdx.x);
        for (; c + 3 * kReadThreads < end; c += 4 * kReadThreads) {
            const auto v0 = f(c), v1 = f(c + kReadThreads), v2 = f(c + 2 * kReadThreads), v3 = f(c + 3 * kReadThreads);
            g(c, v0);
            g(c + kReadThreads, v1);
            g(c + 2 * kReadThreads, v2);
            g(c + 3 * kReadThreads, v3);
        }
        for (; c < end; c += kReadThreads) g(c, f(c));
    }
    // N sums of f(column) over the row, four columns' values added before they meet the sum
    template <int N, class F>
    __device__ __forceinline__ void sums(F&& f, float (&out)[N]) {
        LongSum s[N];
        int c = begin + static_cast<int>(threadIdx.x);
        for (; c + 3 * kReadThreads < end; c += 4 * kReadThreads) {
            const Values<N> v0 = f(c), v1 = f(c + kReadThreads), v2 = f(c + 2 * kReadThreads), v3 = f(c + 3 * kReadThreads);
#pragma unroll
            for (int i = 0; i < N; ++i) s[i].add((v0.v[i] + v1.v[i]) + (v2.v[i] + v3.v[i]));
        }
        for (; c < end; c += kReadThreads) {
            const Values<N> v = f(c);
#pragma unroll
            for (int i = 0; i < N; ++i) s[i].add(v.v[i]);
        }
        const int lane = threadIdx.x & 31;
        cg::cluster_group cl = cg::this_cluster();
        const int n = static_cast<int>(cl.num_blocks()), rank = static_cast<int>(cl.block_rank());
#pragma unroll
        for (int i = 0; i < N; ++i) {
            out[i] = warp_allreduce<SumOp, 32>(s[i].value());
            if (lane == 0) warp[buf][i][threadIdx.x >> 5] = out[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) out[i] = warp_allreduce<SumOp, 32>(lane < kWarps ? warp[buf][i][lane] : 0.0f);
        if (n > 1) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (static_cast<int>(threadIdx.x) < n) *cl.map_shared_rank(&cta[buf][i][rank], threadIdx.x) = out[i];
            cl.sync();
#pragma unroll
            for (int i = 0; i < N; ++i) out[i] = warp_allreduce<SumOp, 32>(lane < n ? cta[buf][i][lane] : 0.0f);
        }
        buf ^= 1;
    }
};

// cp.async: 16 bytes to shared memory past the registers and L1.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// A barrier of one team's threads (a team of one warp needs no more than the warp's own).
__device__ __forceinline__ void team_barrier(int team, int warps) {
    if (warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(warps * 32) : "memory");
}

}  // namespace block
}  // namespace tr
