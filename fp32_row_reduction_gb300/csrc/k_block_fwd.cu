// The gated residual norm, forward: h = rs x + bs gate post(a), y = pre(h).
//
// Each row needs the statistics of a before h exists, and those of h before y:
// two dependent row sums. Rows that fit the chip take tr_block_fwd.cuh's kernel.
#include <algorithm>

#include "tr_block.cuh"
#include "tr_block.h"
#include "tr_launch.h"

namespace tr {
namespace block {

// Rows of any length, type and alignment: a CTA or, for few long rows, a cluster to a row, which is read again
// (from the caches) for each pass.
template <class T, bool LAYER>
__global__ void __launch_bounds__(kReadThreads) fwd_read_kernel(const BlockArgs p) {
    __shared__ ReadRow::WarpSums warp_sums[2];
    __shared__ ReadRow::CtaSums cta_sums[2];
    pdl_enter();
    const int cols = p.cols;
    const float inv_n = 1.0f / static_cast<float>(cols);
    ReadRow rr(cols, warp_sums, cta_sums);
    const int ctas = static_cast<int>(cg::this_cluster().num_blocks());
    const ReadParam post_w(p.post_w, 1), post_b(p.post_b, 0), pre_w(p.pre_w, 1), pre_b(p.pre_b, 0);
    const int start = static_cast<int>(threadIdx.x & 31) % cols;  // the lane's element of a row's start (see lane_mean)
    for (int64_t row = blockIdx.x / ctas; row < p.rows; row += gridDim.x / ctas) {
        const T* xr = static_cast<const T*>(p.x) + row * cols;
        const T* ar = static_cast<const T*>(p.a) + row * cols;
        const ReadParam gate(p.gate ? p.gate + row / p.group_rows * cols : nullptr, 1);
        // mean and 1 / sqrt(mean square about it + eps) of v(column)
        auto statistics = [&](auto&& v, float& mean, float& r) {
            float shift = LAYER ? lane_mean(v(start)) : 0.0f;
            float s[2];
            auto sums_about = [&](float about) {
                rr.sums<2>([&](int c) {
                    const float d = v(c) - about;
                    return Values<2>{{d * d, LAYER ? d : 0.0f}};
                }, s);
            };
            sums_about(shift);
            float off = s[1] * inv_n, squares = s[0];
            if constexpr (LAYER) {
                bool far;
                squares = squares_about_mean(s[0], s[1], off, far);
                if (far) {  // (alike in all threads of the row)
                    shift += off;
                    sums_about(shift);
                    off = s[1] * inv_n;
                    squares = squares_about_mean(s[0], s[1], off, far);
                }
            }
            mean = shift + off;
            r = rsqrtf(fmaf(squares, inv_n, p.eps));
        };
        float ma = 0.0f, ra = 1.0f;
        if (p.post) statistics([&](int c) { return to_float(ar[c]); }, ma, ra);
        auto h_of = [&](int c) {
            const float n = (to_float(ar[c]) - ma) * ra;
            const float scaled = LAYER ? fmaf(n, post_w(c), post_b(c)) : n * post_w(c);
            return p.rs * to_float(xr[c]) + p.bs * (scaled * gate(c));
        };
        float mh = 0.0f, rh = 1.0f;
        if (p.pre) statistics(h_of, mh, rh);
        rr.columns(
            [&](int c) {
                const float h = h_of(c), n = (h - mh) * rh;
                return Values<2>{{h, LAYER ? fmaf(n, pre_w(c), pre_b(c)) : n * pre_w(c)}};
            },
            [&](int c, const Values<2>& v) {
                if (p.h) static_cast<T*>(p.h)[row * cols + c] = from_float<T>(v.v[0]);
                if (p.pre) static_cast<T*>(p.y)[row * cols + c] = from_float<T>(v.v[1]);
            });
    }
    if (ctas > 1) cg::this_cluster().sync();  // no CTA leaves while another may still write to it
}

template <class T, bool LAYER>
cudaError_t fwd_read_launch(const BlockArgs& a, cudaStream_t stream) {
    const int ctas = read_cluster(a.rows, a.cols);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.rows, 1 << 20)) * ctas;
    return launch_dependent(fwd_read_kernel<T, LAYER>, dim3(grid), kReadThreads, 0, ctas, stream, a);
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
