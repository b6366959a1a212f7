// The norm over a list of tensors, and scaling the list by a clipping factor.
//
// A list is cut into tiles of 16 KB; a CTA takes one run of consecutive tiles
// (equal runs, so the split of the sum depends only on the list and the device) and
// walks the tensors its run touches. The norm's CTAs write one partial each, added in
// order by whoever needs the norm.
#include <algorithm>
#include <cstring>

#include "tr_block.cuh"
#include "tr_list.h"

namespace tr {
namespace list {

using block::from_float;
using block::to_float;

constexpr int kUnroll = kListTileBytes / (16 * kListThreads);

// Sum of squares of a thread's elements of one tile, in binary32 where that
// holds them, and again in binary64 from the same registers where it does not. The
// tiles' sums are added in binary64: one such addition for 16 or 32 elements.
struct Squares {
    double total = 0.0;
    template <int M>
    __device__ __forceinline__ void add(const float (&v)[M]) {
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < M; ++i) s[i & 3] = fmaf(v[i], v[i], s[i & 3]);
        const float t = (s[0] + s[1]) + (s[2] + s[3]);
        // t within [2^-96, 2^120]: no square overflowed, and what subnormal squares
        // lost (2^-150 each) is less than 2^-48 of t in all
        if (t >= 0x1p-96f && t <= 0x1p120f) {
            total += static_cast<double>(t);
        } else {
            bool any = false;
#pragma unroll
            for (int i = 0; i < M; ++i) any |= v[i] != 0.0f;
            if (any)
#pragma unroll
                for (int i = 0; i < M; ++i) total += static_cast<double>(v[i]) * static_cast<double>(v[i]);
        }
    }
    __device__ __forceinline__ void merge(double o) { total += o; }
    __device__ __forceinline__ double value() const { return total; }
};

// Largest magnitude, as bits: a NaN's magnitude bits are above infinity's, so a NaN wins.
struct Largest {
    unsigned bits = 0;
    template <int M>
    __device__ __forceinline__ void add(const float (&v)[M]) {
#pragma unroll
        for (int i = 0; i < M; ++i) bits = max(bits, __float_as_uint(v[i]) & 0x7fffffffu);
    }
    __device__ __forceinline__ void merge(double o) {
        bits = max(bits, __float_as_uint(static_cast<float>(o)) & 0x7fffffffu);
    }
    __device__ __forceinline__ double value() const { return static_cast<double>(__uint_as_float(bits)); }
};

// The elements of 16 bytes as floats.
template <class T>
__device__ __forceinline__ void unpack(uint4 q, float (&v)[16 / sizeof(T)]) {
    const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
    for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) v[i] = to_float(e[i]);
}

__device__ __forceinline__ uint4 ld16(const char* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// A tile's elements, kUnroll groups of 16 / sizeof(T) a thread; absent ones are zero.
// base: the tensor's 16-byte boundary; [begin, end): its bytes counted from there.
template <class T>
__device__ __forceinline__ void load_tile(const char* base, int64_t begin, int64_t end, int64_t tile,
                                          float (&v)[kUnroll * 16 / sizeof(T)]) {
    constexpr int E = 16 / sizeof(T);
    uint4 q[kUnroll];
    const int64_t at = tile * kListTileBytes + 16 * static_cast<int64_t>(threadIdx.x);
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
        const int64_t b = at + j * 16 * kListThreads;
        q[j] = make_uint4(0, 0, 0, 0);
        if (b >= begin && b + 16 <= end) {
            q[j] = ld16(base + b);
        } else if (b + 16 > begin && b < end) {
            T* e = reinterpret_cast<T*>(&q[j]);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int64_t bi = b + i * static_cast<int>(sizeof(T));
                if (bi >= begin && bi < end) e[i] = *reinterpret_cast<const T*>(base + bi);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
        float f[E];
        unpack<T>(q[j], f);
#pragma unroll
        for (int i = 0; i < E; ++i) v[j * E + i] = f[i];
    }
}

// f(tensor index, tile of the tensor) for the CTA's run of tiles.
template <int N, class F>
__device__ __forceinline__ void for_run(const TensorList<N>& l, F&& f) {
    const uint32_t tiles = l.first[l.count];
    uint32_t t = static_cast<uint32_t>(static_cast<uint64_t>(tiles) * blockIdx.x / gridDim.x);
    const uint32_t end = static_cast<uint32_t>(static_cast<uint64_t>(tiles) * (blockIdx.x + 1) / gridDim.x);
    int lo = 0, hi = l.count - 1;  // the last tensor that starts at or before t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.first[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    for (; t < end; ++t) {
        while (l.first[lo + 1] <= t) ++lo;
        f(lo, static_cast<int64_t>(t - l.first[lo]));
    }
}

template <class R, int N>
__global__ void __launch_bounds__(kListThreads) norm_kernel(const __grid_constant__ TensorList<N> l, double* part) {
    pdl_enter();
    R r;
    for_run(l, [&](int i, int64_t tile) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(l.in[i]);
        const char* base = reinterpret_cast<const char*>(p & ~static_cast<uintptr_t>(15));
        const int64_t begin = static_cast<int64_t>(p & 15);
        if (l.dtype[i] == TR_F32) {
            float v[kUnroll * 4];
            load_tile<float>(base, begin, begin + l.numel[i] * 4, tile, v);
            r.add(v);
        } else {
            float v[kUnroll * 8];
            if (l.dtype[i] == TR_BF16) load_tile<__nv_bfloat16>(base, begin, begin + l.numel[i] * 2, tile, v);
            else load_tile<__half>(base, begin, begin + l.numel[i] * 2, tile, v);
            r.add(v);
        }
    });
    __shared__ double red[kListThreads / 32];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) r.merge(__shfl_xor_sync(kFull, r.value(), o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = r.value();
    __syncthreads();
    if (threadIdx.x == 0) {
        R t;
        for (int i = 0; i < kListThreads / 32; ++i) t.merge(red[i]);
        part[blockIdx.x] = t.value();
    }
}

// The norm from n partials, in every thread of the CTA.
template <class R>
__device__ __forceinline__ double total_of(const double* part, int n, double* red) {
    R r;
    for (int i = threadIdx.x; i < n; i += kListThreads) r.merge(part[i]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) r.merge(__shfl_xor_sync(kFull, r.value(), o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = r.value();
    __syncthreads();
    R t;
#pragma unroll
    for (int i = 0; i < kListThreads / 32; ++i) t.merge(red[i]);
    return t.value();
}
__device__ __forceinline__ float norm_of(int kind, const double* part, int n) {
    __shared__ double red[kListThreads / 32];
    if (kind == TR_TOTAL_L2) return static_cast<float>(sqrt(total_of<Squares>(part, n, red)));
    return static_cast<float>(total_of<Largest>(part, n, red));
}

__global__ void __launch_bounds__(kListThreads) total_kernel(int kind, const double* part, int n, float* norm) {
    pdl_enter();
    const float t = norm_of(kind, part, n);
    if (threadIdx.x == 0) *norm = t;
}

template <class T>
__device__ __forceinline__ void scale_tile(const char* in, char* out, int64_t numel, int64_t tile, float f) {
    constexpr int E = 16 / sizeof(T);
    const uintptr_t p = reinterpret_cast<uintptr_t>(in);
    const char* base = reinterpret_cast<const char*>(p & ~static_cast<uintptr_t>(15));
    const int64_t begin = static_cast<int64_t>(p & 15), end = begin + numel * static_cast<int64_t>(sizeof(T));
    float v[kUnroll * E];
    load_tile<T>(base, begin, end, tile, v);
    char* to = out - begin;
    const bool phase = ((reinterpret_cast<uintptr_t>(out) ^ p) & 15) == 0;
    const int64_t at = tile * kListTileBytes + 16 * static_cast<int64_t>(threadIdx.x);
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
        const int64_t b = at + j * 16 * kListThreads;
        uint4 q;
        T* e = reinterpret_cast<T*>(&q);
#pragma unroll
        for (int i = 0; i < E; ++i) e[i] = from_float<T>(v[j * E + i] * f);
        if (phase && b >= begin && b + 16 <= end) {
            *reinterpret_cast<uint4*>(to + b) = q;
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int64_t bi = b + i * static_cast<int>(sizeof(T));
                if (bi >= begin && bi < end) *reinterpret_cast<T*>(to + bi) = e[i];
            }
        }
    }
}

template <int N>
__global__ void __launch_bounds__(kListThreads)
    scale_kernel(const __grid_constant__ TensorList<N> l, int kind, const double* part, int n, float* norm, int write,
                 float max_norm, float eps) {
    pdl_enter();
    const float total = n > 0 ? norm_of(kind, part, n) : *norm;
    if (write && blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    const float ratio = max_norm / (total + eps);
    const float f = ratio > 1.0f ? 1.0f : ratio;  // a NaN stays
    for_run(l, [&](int i, int64_t tile) {
        if (l.dtype[i] == TR_F32) scale_tile<float>(l.in[i], l.out[i], l.numel[i], tile, f);
        else if (l.dtype[i] == TR_BF16) scale_tile<__nv_bfloat16>(l.in[i], l.out[i], l.numel[i], tile, f);
        else scale_tile<__half>(l.in[i], l.out[i], l.numel[i], tile, f);
    });
}

template <class Dst, class Src>
void copy_list(Dst* d, const Src& s) {
    d->count = s.count;
    std::memcpy(d->in, s.in, sizeof(s.in[0]) * s.count);
    std::memcpy(d->out, s.out, sizeof(s.out[0]) * s.count);
    std::memcpy(d->numel, s.numel, sizeof(s.numel[0]) * s.count);
    std::memcpy(d->first, s.first, sizeof(s.first[0]) * (s.count + 1));
    std::memcpy(d->dtype, s.dtype, s.count);
}

// CTAs of a launch: what the device holds at once, but no more than there are tiles.
int list_ctas(const void* kernel, uint32_t tiles) {
    int dev = 0, sms = 0, per = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kListThreads, 0) != cudaSuccess)
        return 0;
    return static_cast<int>(std::min<int64_t>(tiles, std::min(kListMaxCtas, std::max(1, per) * sms)));
}

template <class R>
cudaError_t norm_launch(const TensorList<kListMax>& l, double* part, int* ctas, cudaStream_t stream) {
    *ctas = list_ctas(reinterpret_cast<const void*>(norm_kernel<R, kListMax>), l.first[l.count]);
    if (*ctas < 1) return cudaGetLastError();
    if (l.count <= kListFew) {
        TensorList<kListFew> few;
        copy_list(&few, l);
        norm_kernel<R, kListFew><<<*ctas, kListThreads, 0, stream>>>(few, part);
    } else {
        norm_kernel<R, kListMax><<<*ctas, kListThreads, 0, stream>>>(l, part);
    }
    return cudaGetLastError();
}

}  // namespace list

cudaError_t launch_list_norm(int kind, const TensorList<kListMax>& l, double* part, int* ctas, cudaStream_t stream) {
    return kind == TR_TOTAL_L2 ? list::norm_launch<list::Squares>(l, part, ctas, stream)
                               : list::norm_launch<list::Largest>(l, part, ctas, stream);
}

cudaError_t launch_list_total(int kind, const double* part, int n, float* norm, cudaStream_t stream) {
    list::total_kernel<<<1, kListThreads, 0, stream>>>(kind, part, n, norm);
    return cudaGetLastError();
}

cudaError_t launch_list_scale(int kind, const TensorList<kListMax>& l, const double* part, int n, float* norm, int write,
                              float max_norm, float eps, cudaStream_t stream) {
    const int ctas = list::list_ctas(reinterpret_cast<const void*>(list::scale_kernel<kListMax>), l.first[l.count]);
    if (ctas < 1) return cudaGetLastError();
    if (l.count <= kListFew) {
        TensorList<kListFew> few;
        list::copy_list(&few, l);
        list::scale_kernel<kListFew><<<ctas, kListThreads, 0, stream>>>(few, kind, part, n, norm, write, max_norm, eps);
    } else {
        list::scale_kernel<kListMax><<<ctas, kListThreads, 0, stream>>>(l, kind, part, n, norm, write, max_norm, eps);
    }
    return cudaGetLastError();
}

}  // namespace tr
