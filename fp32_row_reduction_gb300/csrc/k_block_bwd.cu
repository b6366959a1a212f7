// The gated residual norm, backward. With hh = (h - mean h) r_h, u = dy w,
// ah = (a - mean a) r_a and q = bs gate D w_post (RMSNorm: means 0, and no mean
// terms below):
//   D  = dh + r_h (u - mean u - hh mean(u hh)),  dx = rs D
//   da = r_a (q - mean q - ah mean(q ah))        (no post-norm: da = bs gate D)
//   dw = sum dy hh, db = sum dy over the rows
//   dw_post = bs sum gate D ah, db_post = bs sum gate D
//   dgate = bs (w_post sum D ah + b_post sum D) over the gate row's own rows
//           (no post-norm: bs sum D a)
// so two column sums a norm (one for RMSNorm) serve all five column gradients:
// where a slab's rows share a gate row, sum D ah and sum D give dgate, dw_post and
// db_post alike. Slabs of rows sum their columns apart; a last kernel adds the slabs in order.
#include <algorithm>

#include "tr_block.cuh"
#include "tr_block.h"
#include "tr_launch.h"

namespace tr {
namespace block {

constexpr int kReadThreads = 512;
constexpr int kTile = 32;  // columns of a column-sum CTA

// ---- rows of any length, type and alignment, read again for each pass ----------

// dx, da and the row's statistics.
template <class T, bool LAYER>
__global__ void __launch_bounds__(kReadThreads) bwd_read_kernel(const BlockBwArgs p) {
    constexpr int W = kReadThreads / 32;
    __shared__ float slot[2][W];
    pdl_enter();
    int buf = 0;
    const int cols = p.cols;
    const float n = static_cast<float>(cols);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const int64_t at = row * cols;
        const T* hr = static_cast<const T*>(p.h) + at;
        const T* ar = static_cast<const T*>(p.a) + at;
        const T* dyr = static_cast<const T*>(p.dy) + at;
        const T* dhr = p.dh ? static_cast<const T*>(p.dh) + at : nullptr;
        const float* gr = p.gate ? p.gate + row / p.group_rows * cols : nullptr;
        auto mean_of = [&](auto&& f) {
            LongSum s;
            for (int c = threadIdx.x; c < cols; c += kReadThreads) s.add(f(c));
            float v[1] = {s.value()};
            cta_sums<1, W>(v, slot, buf);
            return v[0] / n;
        };
        auto statistics = [&](const T* v, float& mean, float& r) {
            mean = LAYER ? mean_of([&](int c) { return to_float(v[c]); }) : 0.0f;
            const float m = mean;
            r = 1.0f / sqrtf(mean_of([&](int c) {
                const float d = to_float(v[c]) - m;
                return d * d;
            }) + p.eps);
        };
        float mh = 0.0f, rh = 0.0f, c1 = 0.0f, c2 = 0.0f, ma = 0.0f, ra = 0.0f;
        auto u_of = [&](int c) { return to_float(dyr[c]) * (p.pre_w ? __ldg(p.pre_w + c) : 1.0f); };
        auto hh_of = [&](int c) { return (to_float(hr[c]) - mh) * rh; };
        auto ah_of = [&](int c) { return (to_float(ar[c]) - ma) * ra; };
        if (p.pre) {
            statistics(hr, mh, rh);
            if (LAYER) c1 = mean_of(u_of);
            c2 = mean_of([&](int c) { return u_of(c) * hh_of(c); });
        }
        auto d_of = [&](int c) {
            float d = dhr ? to_float(dhr[c]) : 0.0f;
            if (p.pre) d += rh * (u_of(c) - c1 - hh_of(c) * c2);
            return d;
        };
        auto q_of = [&](float d, int c) {
            float q = p.bs * d;
            if (gr) q *= __ldg(gr + c);
            if (p.post && p.post_w) q *= __ldg(p.post_w + c);
            return q;
        };
        float e1 = 0.0f, e2 = 0.0f;
        if (p.post) {
            statistics(ar, ma, ra);
            if (LAYER) e1 = mean_of([&](int c) { return q_of(d_of(c), c); });
            e2 = mean_of([&](int c) { return q_of(d_of(c), c) * ah_of(c); });
        }
        if (p.sums && threadIdx.x == 0) {
            float* s = p.stats + row * kBlockStats;
            s[0] = mh;
            s[1] = rh;
            s[2] = c1;
            s[3] = c2;
            s[4] = ma;
            s[5] = ra;
        }
        for (int c = threadIdx.x; c < cols; c += kReadThreads) {
            const float d = d_of(c);
            const float q = q_of(d, c);
            static_cast<T*>(p.dx)[at + c] = from_float<T>(p.rs * d);
            static_cast<T*>(p.da)[at + c] = from_float<T>(p.post ? ra * (q - e1 - ah_of(c) * e2) : q);
        }
    }
}

// The column sums of one slab over kTile columns, from the rows' statistics:
// 8 rows at a time, one a warp.
template <class T, bool LAYER>
__global__ void __launch_bounds__(kTile * 8) bwd_columns_kernel(const BlockBwArgs p) {
    constexpr int V = LAYER ? 4 : 2;
    __shared__ float red[8][V][kTile];
    pdl_enter();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int cols = p.cols;
    const int c = static_cast<int>(blockIdx.x) * kTile + lane;
    const bool ok = c < cols;
    const SlabRows rows = slab_rows(p, blockIdx.y);
    const float pw = ok && p.pre_w ? p.pre_w[c] : 1.0f;
    const float ow = ok && p.post && p.post_w ? p.post_w[c] : 1.0f;
    const float ob = ok && p.post && p.post_b ? p.post_b[c] : 0.0f;
    const bool need_a = p.post || p.dgate;
    LongSum pre0, pre1;      // dy hh, dy
    float out0 = 0.0f, out1 = 0.0f;  // whole groups: sums of gate D ah, gate D
    int64_t row = rows.begin;
    while (row < rows.end) {
        const int64_t end = p.slices > 0 ? rows.end : row + p.group_rows;
        LongSum a0, a1;  // D ah, D of one gate row
        for (int64_t r = row + w; r < end; r += 8) {
            if (!ok) continue;
            const float* s = p.stats + r * kBlockStats;
            const int64_t at = r * cols + c;
            float d = p.dh ? to_float(static_cast<const T*>(p.dh)[at]) : 0.0f;
            if (p.pre) {
                const float dy = to_float(static_cast<const T*>(p.dy)[at]);
                const float hh = (to_float(static_cast<const T*>(p.h)[at]) - s[0]) * s[1];
                d += s[1] * (dy * pw - s[2] - hh * s[3]);
                pre0.add(dy * hh);
                if (LAYER) pre1.add(dy);
            }
            if (need_a) {
                const float v = to_float(static_cast<const T*>(p.a)[at]);
                a0.add(d * (p.post ? (v - s[4]) * s[5] : v));
                if (LAYER) a1.add(d);
            }
        }
        if (p.slices > 0) {
            out0 = a0.value();
            out1 = a1.value();
            break;
        }
        // one whole group: its gate gradient is final
        red[w][0][lane] = a0.value();
        if (LAYER) red[w][1][lane] = a1.value();
        __syncthreads();
        if (w == 0) {
            float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s0 += red[i][0][lane];
                if (LAYER) s1 += red[i][1][lane];
            }
            if (ok) {
                const int64_t g = row / p.group_rows;
                const float gate = p.gate[g * cols + c];
                if (p.dgate) p.dgate[g * cols + c] = p.bs * (ow * s0 + ob * s1);
                out0 += gate * s0;
                out1 += gate * s1;
            }
        }
        __syncthreads();
        row = end;
    }
    red[w][0][lane] = pre0.value();
    red[w][1][lane] = out0;
    if (LAYER) {
        red[w][2 % V][lane] = pre1.value();
        red[w][3 % V][lane] = out1;
    }
    __syncthreads();
    if (w < V && ok) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += red[i][w][lane];
        p.part[(static_cast<int64_t>(blockIdx.y) * V + w) * cols + c] = s;
    }
}

// ---- the slabs' partials to the column gradients --------------------------------

// kTile columns a CTA, 32 warps. Warp w adds slabs w, w + 32, ...; with slices the
// warps first share out the groups, `per` (a power of two) warps to a group.
template <bool LAYER>
__global__ void __launch_bounds__(1024) bwd_finish_kernel(const BlockBwArgs p) {
    constexpr int V = LAYER ? 4 : 2;
    __shared__ float red[32][2][kTile];
    pdl_enter();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int cols = p.cols;
    const int c = static_cast<int>(blockIdx.x) * kTile + lane;
    const bool ok = c < cols;
    auto part = [&](int64_t s, int v) { return ok ? p.part[(s * V + v) * cols + c] : 0.0f; };
    auto total = [&](float v0, float v1, float& t0, float& t1) {  // over the warps, for warp 0
        red[w][0][lane] = v0;
        red[w][1][lane] = v1;
        __syncthreads();
        t0 = t1 = 0.0f;
        if (w == 0)
#pragma unroll 8
            for (int i = 0; i < 32; ++i) {
                t0 += red[i][0][lane];
                t1 += red[i][1][lane];
            }
        __syncthreads();
    };
    if (p.pre) {
        float s0 = 0.0f, s1 = 0.0f, t0, t1;
        for (int64_t s = w; s < p.slabs; s += 32) {
            s0 += part(s, 0);
            if (LAYER) s1 += part(s, 2 % V);
        }
        total(s0, s1, t0, t1);
        if (w == 0 && ok) {
            if (p.dpre_w) p.dpre_w[c] = t0;
            if (LAYER && p.dpre_b) p.dpre_b[c] = t1;
        }
    }
    if (!p.post && !p.dgate) return;
    const float ow = ok && p.post && p.post_w ? p.post_w[c] : 1.0f;
    const float ob = ok && p.post && p.post_b ? p.post_b[c] : 0.0f;
    float x0 = 0.0f, x1 = 0.0f;  // gate D ah, gate D
    if (p.slices == 0) {
        for (int64_t s = w; s < p.slabs; s += 32) {
            x0 += part(s, 1);
            if (LAYER) x1 += part(s, 3 % V);
        }
    } else {
        int per = 32;
        while (per > 1 && 32 / per < p.groups) per >>= 1;
        const int at_once = 32 / per, mine = w / per, sub = w % per;
        for (int64_t g0 = 0; g0 < p.groups; g0 += at_once) {
            const int64_t g = g0 + mine;
            float s0 = 0.0f, s1 = 0.0f;
            if (g < p.groups)
                for (int64_t i = sub; i < p.slices; i += per) {
                    s0 += part(g * p.slices + i, 1);
                    if (LAYER) s1 += part(g * p.slices + i, 3 % V);
                }
            red[w][0][lane] = s0;
            red[w][1][lane] = s1;
            __syncthreads();
            if (sub == 0 && g < p.groups && ok) {
                s0 = s1 = 0.0f;
                for (int i = 0; i < per; ++i) {
                    s0 += red[w + i][0][lane];
                    s1 += red[w + i][1][lane];
                }
                if (p.dgate) p.dgate[g * cols + c] = p.bs * (ow * s0 + ob * s1);
                const float gate = p.gate ? p.gate[g * cols + c] : 1.0f;
                x0 += gate * s0;
                x1 += gate * s1;
            }
            __syncthreads();
        }
    }
    float t0, t1;
    total(x0, x1, t0, t1);
    if (w == 0 && ok && p.post) {
        if (p.dpost_w) p.dpost_w[c] = p.bs * t0;
        if (LAYER && p.dpost_b) p.dpost_b[c] = p.bs * t1;
    }
}

template <class T, bool LAYER>
cudaError_t bwd_launch(const BlockBwArgs& in, cudaStream_t stream) {
    BlockBwArgs a = in;
    block_slabs(&a, block_slab_limit(a.rows, a.cols));
    const unsigned tiles = static_cast<unsigned>((a.cols + kTile - 1) / kTile);
    bwd_read_kernel<T, LAYER><<<static_cast<unsigned>(std::min<int64_t>(a.rows, 1 << 20)), kReadThreads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.sums) return e;
    bwd_columns_kernel<T, LAYER><<<dim3(tiles, static_cast<unsigned>(a.slabs)), kTile * 8, 0, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_block_finish(LAYER ? TR_NORM_LAYER : TR_NORM_RMS, a, stream);
}

template <class T>
cudaError_t bwd_read(int kind, const BlockBwArgs& a, cudaStream_t stream) {
    return kind == TR_NORM_LAYER ? bwd_launch<T, true>(a, stream) : bwd_launch<T, false>(a, stream);
}

}  // namespace block

cudaError_t launch_block_finish(int kind, const BlockBwArgs& a, cudaStream_t stream) {
    const dim3 tiles(static_cast<unsigned>((a.cols + block::kTile - 1) / block::kTile));
    return kind == TR_NORM_LAYER ? launch_dependent(block::bwd_finish_kernel<true>, tiles, 1024, 0, 1, stream, a)
                                 : launch_dependent(block::bwd_finish_kernel<false>, tiles, 1024, 0, 1, stream, a);
}

cudaError_t launch_block_backward(int kind, int dtype, const BlockBwArgs& a, cudaStream_t stream) {
    bool done = false;
    cudaError_t e = cudaErrorInvalidValue;
    switch (dtype) {
        case TR_F32:
            e = launch_block_backward_f32(kind, a, &done, stream);
            return done ? e : block::bwd_read<float>(kind, a, stream);
        case TR_BF16:
            e = launch_block_backward_bf16(kind, a, &done, stream);
            return done ? e : block::bwd_read<__nv_bfloat16>(kind, a, stream);
        case TR_F16:
            e = launch_block_backward_f16(kind, a, &done, stream);
            return done ? e : block::bwd_read<__half>(kind, a, stream);
    }
    return e;
}

}  // namespace tr
