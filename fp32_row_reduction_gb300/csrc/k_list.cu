// The norm over a list of tensors, and scaling the list by a clipping factor.
//
// A list is cut into tiles of 16 KB; a CTA takes one run of consecutive tiles
// (equal runs, so the split of the sum depends only on the list and the device) and
// walks the tensors its run touches. The norm's CTAs write one partial each, added in
// order by whoever needs the norm. Both passes wait for memory: the norm of 1.41 GB in 121 tensors takes
// 207 us (6.8 TB/s), with the scaling into other tensors 650 us (6.5 TB/s over the three passes).
#include <algorithm>
#include <cstring>

#include "tr_block.cuh"
#include "tr_launch.h"
#include "tr_list.h"

namespace tr {
namespace list {

using block::from_float;
using block::to_float;

// What the norm's pass asks L2 to keep for the scaling pass, in all. Of 86 MB of float32: 42 us with 80 or 96 MB,
// 44 with 64, 48 with 32, 46 with none asked for (a 126 MB cache in two halves).
constexpr int64_t kListKeepBytes = 80LL << 20;
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

// Where a tile of a tensor lies: `base` is the tensor's 16-byte boundary, [begin, end) its bytes from there.
struct Place {
    const char* base;
    int64_t begin, end, at;  // at: this thread's first byte of the tile
    bool whole;              // all of the tile is in the tensor
};
template <int N>
__device__ __forceinline__ Place place_of(const TensorList<N>& l, int i, uint32_t t) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(l.in[i]);
    const int64_t tile = static_cast<int64_t>(t - l.first[i]) * kListTileBytes;
    Place q;
    q.base = reinterpret_cast<const char*>(p & ~static_cast<uintptr_t>(15));
    q.begin = static_cast<int64_t>(p & 15);
    q.end = q.begin + l.numel[i] * (l.dtype[i] == TR_F32 ? 4 : 2);
    q.at = tile + 16 * static_cast<int64_t>(threadIdx.x);
    q.whole = tile >= q.begin && tile + kListTileBytes <= q.end;
    return q;
}

// How L2 is to treat a load: nothing said, kept for a second use, or last use.
enum Keep : int { KEEP_PLAIN, KEEP_LAST, KEEP_FIRST };
struct Policies {
    uint64_t last, first;
    __device__ __forceinline__ Policies() {
        asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(last));
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
    }
};
__device__ __forceinline__ uint4 ld16(const char* p, const Policies& pol, int keep) {
    uint4 v;
    if (keep == KEEP_PLAIN) {
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(p)
                     : "memory");
    } else {
        asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(p), "l"(keep == KEEP_LAST ? pol.last : pol.first)
                     : "memory");
    }
    return v;
}

// A thread's 16-byte words of a tile; elements outside the tensor (of 2 or 4 bytes) are zero.
__device__ __forceinline__ void load_tile(const Place& p, int size, const Policies& pol, int keep, uint4 (&q)[kUnroll]) {
    if (p.whole) {
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) q[j] = ld16(p.base + p.at + j * 16 * kListThreads, pol, keep);
        return;
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
        const int64_t b = p.at + j * 16 * kListThreads;
        q[j] = make_uint4(0, 0, 0, 0);
        if (b >= p.begin && b + 16 <= p.end) {
            q[j] = ld16(p.base + b, pol, keep);
        } else if (b + 16 > p.begin && b < p.end) {
            uint32_t* word = reinterpret_cast<uint32_t*>(&q[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t bi = b + 4 * i;
                if (size == 4) {
                    if (bi >= p.begin && bi < p.end) word[i] = *reinterpret_cast<const uint32_t*>(p.base + bi);
                } else {
                    if (bi >= p.begin && bi < p.end) word[i] = *reinterpret_cast<const uint16_t*>(p.base + bi);
                    if (bi + 2 >= p.begin && bi + 2 < p.end)
                        word[i] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p.base + bi + 2)) << 16;
                }
            }
        }
    }
}

// The elements of 16 bytes as floats.
template <class T>
__device__ __forceinline__ void unpack(const uint4 (&q)[kUnroll], float (&v)[kUnroll * 16 / sizeof(T)]) {
    constexpr int E = 16 / sizeof(T);
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
        const T* e = reinterpret_cast<const T*>(&q[j]);
#pragma unroll
        for (int i = 0; i < E; ++i) v[j * E + i] = to_float(e[i]);
    }
}

// The CTA's run of tiles, in order or from its end: the next tile's words are on their way while
// f(tensor, place, words) works on one.
// The last `keep` tiles of every run are loaded to stay in L2 (forward), and the others are not; backward every load
// is the last.
template <bool BACKWARD, int N, class F>
__device__ __forceinline__ void for_run(const TensorList<N>& l, uint32_t keep, F&& f) {
    const Policies pol;
    const uint32_t tiles = l.first[l.count];
    const uint32_t begin = static_cast<uint32_t>(static_cast<uint64_t>(tiles) * blockIdx.x / gridDim.x);
    const uint32_t end = static_cast<uint32_t>(static_cast<uint64_t>(tiles) * (blockIdx.x + 1) / gridDim.x);
    if (begin >= end) return;
    uint32_t t = BACKWARD ? end - 1 : begin;
    int lo = 0, hi = l.count - 1;  // the last tensor that starts at or before t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.first[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    uint4 q[kUnroll];
    Place p = place_of(l, lo, t);
    auto treat = [&](uint32_t left) { return BACKWARD ? KEEP_FIRST : keep == 0 ? KEEP_PLAIN : left <= keep ? KEEP_LAST : KEEP_FIRST; };
    load_tile(p, l.dtype[lo] == TR_F32 ? 4 : 2, pol, treat(end - begin), q);
    for (uint32_t n = end - begin; n > 0; --n) {
        uint4 ahead[kUnroll];
        const int i = lo;
        Place next = p;
        if (n > 1) {
            if (BACKWARD) {
                --t;
                while (l.first[lo] > t) --lo;
            } else {
                ++t;
                while (l.first[lo + 1] <= t) ++lo;
            }
            next = place_of(l, lo, t);
            load_tile(next, l.dtype[lo] == TR_F32 ? 4 : 2, pol, treat(n - 1), ahead);
        }
        f(i, p, q);
        p = next;
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) q[j] = ahead[j];
    }
}

template <class R, int N>
__global__ void __launch_bounds__(kListThreads) norm_kernel(const __grid_constant__ TensorList<N> l, double* part, uint32_t keep) {
    pdl_enter();
    R r;
    for_run<false>(l, keep, [&](int i, const Place&, const uint4 (&q)[kUnroll]) {
        if (l.dtype[i] == TR_F32) {
            float v[kUnroll * 4];
            unpack<float>(q, v);
            r.add(v);
        } else {
            float v[kUnroll * 8];
            if (l.dtype[i] == TR_BF16) unpack<__nv_bfloat16>(q, v);
            else unpack<__half>(q, v);
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

// A tile scaled into `out`. Where out has another place within 16 bytes than in, the tile goes element by
// element, neighbours to neighbours: 2 or 4 bytes a lane, but whole sectors.
template <class T>
__device__ __forceinline__ void scale_tile(const char* in, char* out, const Place& p, const uint4 (&q)[kUnroll], float f) {
    constexpr int E = 16 / sizeof(T);
    if (((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(in)) & 15) != 0) {
        const T* from = reinterpret_cast<const T*>(in);
        T* to = reinterpret_cast<T*>(out);
        const int64_t n = (p.end - p.begin) / static_cast<int64_t>(sizeof(T));
        const int64_t first = (p.at - 16 * static_cast<int64_t>(threadIdx.x) - p.begin) / static_cast<int64_t>(sizeof(T)) + threadIdx.x;
#pragma unroll 8
        for (int k = 0; k < kUnroll * E; ++k) {
            const int64_t e = first + k * kListThreads;
            if (e >= 0 && e < n) to[e] = from_float<T>(to_float(from[e]) * f);
        }
        return;
    }
    float v[kUnroll * E];
    unpack<T>(q, v);
    char* to = out - p.begin + p.at;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
        const int64_t b = p.at + j * 16 * kListThreads;
        uint4 o;
        T* e = reinterpret_cast<T*>(&o);
#pragma unroll
        for (int i = 0; i < E; ++i) e[i] = from_float<T>(v[j * E + i] * f);
        if (p.whole || (b >= p.begin && b + 16 <= p.end)) {
            __stcs(reinterpret_cast<uint4*>(to + j * 16 * kListThreads), o);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int64_t bi = b + i * static_cast<int>(sizeof(T));
                if (bi >= p.begin && bi < p.end) reinterpret_cast<T*>(to + j * 16 * kListThreads)[i] = e[i];
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
    // from the end of the run, which the norm's pass read last
    for_run<true>(l, 0, [&](int i, const Place& p, const uint4 (&q)[kUnroll]) {
        if (l.dtype[i] == TR_F32) scale_tile<float>(l.in[i], l.out[i], p, q, f);
        else if (l.dtype[i] == TR_BF16) scale_tile<__nv_bfloat16>(l.in[i], l.out[i], p, q, f);
        else scale_tile<__half>(l.in[i], l.out[i], p, q, f);
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
    return static_cast<int>(std::min<int64_t>(tiles, std::min(kListMaxCtas, resident_ctas(kernel, kListThreads, 0))));
}

template <class R>
cudaError_t norm_launch(const TensorList<kListMax>& l, double* part, bool again, int* ctas, cudaStream_t stream) {
    const uint32_t tiles = l.first[l.count];
    *ctas = list_ctas(reinterpret_cast<const void*>(norm_kernel<R, kListMax>), tiles);
    if (*ctas < 1) return cudaErrorInvalidConfiguration;
    // what is kept of each run for the scaling pass
    const uint32_t keep = again ? std::max<uint32_t>(1, static_cast<uint32_t>(std::min<int64_t>(tiles, kListKeepBytes / kListTileBytes) / *ctas)) : 0;
    if (l.count <= kListFew) {
        TensorList<kListFew> few;
        copy_list(&few, l);
        return launch_dependent(norm_kernel<R, kListFew>, dim3(*ctas), kListThreads, 0, 1, stream, few, part, keep);
    }
    return launch_dependent(norm_kernel<R, kListMax>, dim3(*ctas), kListThreads, 0, 1, stream, l, part, keep);
}

}  // namespace list

cudaError_t launch_list_norm(int kind, const TensorList<kListMax>& l, double* part, bool again, int* ctas, cudaStream_t stream) {
    return kind == TR_TOTAL_L2 ? list::norm_launch<list::Squares>(l, part, again, ctas, stream)
                               : list::norm_launch<list::Largest>(l, part, again, ctas, stream);
}

cudaError_t launch_list_total(int kind, const double* part, int n, float* norm, cudaStream_t stream) {
    return launch_dependent(list::total_kernel, dim3(1), kListThreads, 0, 1, stream, kind, part, n, norm);
}

cudaError_t launch_list_scale(int kind, const TensorList<kListMax>& l, const double* part, int n, float* norm, int write,
                              float max_norm, float eps, cudaStream_t stream) {
    const int ctas = list::list_ctas(reinterpret_cast<const void*>(list::scale_kernel<kListMax>), l.first[l.count]);
    if (ctas < 1) return cudaErrorInvalidConfiguration;
    if (l.count <= kListFew) {
        TensorList<kListFew> few;
        list::copy_list(&few, l);
        return launch_dependent(list::scale_kernel<kListFew>, dim3(ctas), kListThreads, 0, 1, stream, few, kind, part, n, norm, write, max_norm, eps);
    }
    return launch_dependent(list::scale_kernel<kListMax>, dim3(ctas), kListThreads, 0, 1, stream, l, kind, part, n, norm, write, max_norm, eps);
}

}  // namespace tr
