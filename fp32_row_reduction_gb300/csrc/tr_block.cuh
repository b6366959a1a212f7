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

// A long sum in two levels: binary32 over 32 terms at a time, their totals in
// binary64, so that a row of 2^24 columns loses no more than a short one.
struct LongSum {
    float part = 0.0f;
    double total = 0.0;
    int n = 0;
    __device__ __forceinline__ void add(float v) {
        part += v;
        if (++n == 32) {
            total += static_cast<double>(part);
            part = 0.0f;
            n = 0;
        }
    }
    __device__ __forceinline__ float value() const { return static_cast<float>(total + static_cast<double>(part)); }
};

// N sums over a CTA of WARPS warps in one exchange (every thread gets them).
// `buf` alternates between the halves of `slot`, so consecutive sums need one barrier each.
template <int N, int WARPS>
__device__ __forceinline__ void cta_sums(float (&v)[N], float (*slot)[N * WARPS], int& buf) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kFull, v[i], o);
    float* s = slot[buf];
    buf ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) s[i * WARPS + (threadIdx.x >> 5)] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float t = lane < WARPS ? s[i * WARPS + lane] : 0.0f;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(kFull, t, o);
        v[i] = t;
    }
}

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
