// The gated residual norm, forward: h = rs x + bs gate post(a), y = pre(h).
//
// Each row needs the statistics of a before h exists, and those of h before y:
// two dependent row sums (LayerNorm: four, each variance about its mean).
#include <algorithm>

#include "tr_block.cuh"
#include "tr_block.h"

namespace tr {
namespace block {

constexpr int kReadThreads = 512;

// Rows of any length, type and alignment: a CTA per row, the row read again (from
// the caches) for each pass.
template <class T, bool LAYER>
__global__ void __launch_bounds__(kReadThreads) fwd_read_kernel(const BlockArgs p) {
    constexpr int W = kReadThreads / 32;
    __shared__ float slot[2][W];
    pdl_enter();
    int buf = 0;
    const int cols = p.cols;
    const float n = static_cast<float>(cols);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* xr = static_cast<const T*>(p.x) + row * cols;
        const T* ar = static_cast<const T*>(p.a) + row * cols;
        const float* gr = p.gate ? p.gate + row / p.group_rows * cols : nullptr;
        auto row_sum = [&](auto&& f) {
            LongSum s;
            for (int c = threadIdx.x; c < cols; c += kReadThreads) s.add(f(c));
            float v[1] = {s.value()};
            cta_sums<1, W>(v, slot, buf);
            return v[0];
        };
        // mean and 1 / sqrt(mean square about it + eps) of v(c)
        auto statistics = [&](auto&& v, float& mean, float& r) {
            mean = LAYER ? row_sum(v) / n : 0.0f;
            const float m = mean;
            const float var = row_sum([&](int c) {
                const float d = v(c) - m;
                return d * d;
            }) / n;
            r = 1.0f / sqrtf(var + p.eps);
        };
        float ma = 0.0f, ra = 1.0f;
        if (p.post) statistics([&](int c) { return to_float(ar[c]); }, ma, ra);
        auto h_of = [&](int c) {
            float v = to_float(ar[c]);
            if (p.post) {
                v = (v - ma) * ra;
                if (p.post_w) v *= __ldg(p.post_w + c);
                if (p.post_b) v += __ldg(p.post_b + c);
            }
            if (gr) v *= __ldg(gr + c);
            return p.rs * to_float(xr[c]) + p.bs * v;
        };
        float mh = 0.0f, rh = 1.0f;
        if (p.pre) statistics(h_of, mh, rh);
        for (int c = threadIdx.x; c < cols; c += kReadThreads) {
            const float h = h_of(c);
            if (p.h) static_cast<T*>(p.h)[row * cols + c] = from_float<T>(h);
            if (p.pre) {
                float y = (h - mh) * rh;
                if (p.pre_w) y *= __ldg(p.pre_w + c);
                if (p.pre_b) y += __ldg(p.pre_b + c);
                static_cast<T*>(p.y)[row * cols + c] = from_float<T>(y);
            }
        }
    }
}

template <class T, bool LAYER>
cudaError_t fwd_read_launch(const BlockArgs& a, cudaStream_t stream) {
    const unsigned ctas = static_cast<unsigned>(std::min<int64_t>(a.rows, 1 << 20));
    fwd_read_kernel<T, LAYER><<<ctas, kReadThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <class T>
cudaError_t fwd_read(int kind, const BlockArgs& a, cudaStream_t stream) {
    return kind == TR_NORM_LAYER ? fwd_read_launch<T, true>(a, stream) : fwd_read_launch<T, false>(a, stream);
}

}  // namespace block

cudaError_t launch_block_forward(int kind, int dtype, const BlockArgs& a, cudaStream_t stream) {
    bool done = false;
    cudaError_t e = cudaErrorInvalidValue;
    switch (dtype) {
        case TR_F32:
            e = launch_block_forward_f32(kind, a, &done, stream);
            return done ? e : block::fwd_read<float>(kind, a, stream);
        case TR_BF16:
            e = launch_block_forward_bf16(kind, a, &done, stream);
            return done ? e : block::fwd_read<__nv_bfloat16>(kind, a, stream);
        case TR_F16:
            e = launch_block_forward_f16(kind, a, &done, stream);
            return done ? e : block::fwd_read<__half>(kind, a, stream);
    }
    return e;
}

}  // namespace tr
