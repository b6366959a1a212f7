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

constexpr int kTile = 32;  // columns of a column-sum CTA

// ---- rows of any length, type and alignment, read again for each pass ----------

// dx, da and the row's statistics.
template <class T, bool LAYER, bool PRE, bool POST>
__global__ void __launch_bounds__(kReadThreads) bwd_read_kernel(const BlockBwArgs p) {
    __shared__ ReadRow::WarpSums warp_sums[2];
    __shared__ ReadRow::CtaSums cta_sums[2];
    pdl_enter();
    const int cols = p.cols;
    const float inv_n = 1.0f / static_cast<float>(cols);
    ReadRow rr(cols, warp_sums, cta_sums);
    const int ctas = static_cast<int>(cg::this_cluster().num_blocks());
    const ReadParam pre_w(p.pre_w, 1), post_w(p.post_w, 1);
    const int start = static_cast<int>(threadIdx.x & 31) % cols;  // the lane's element of a row's start (see lane_mean)
    for (int64_t row = blockIdx.x / ctas; row < p.rows; row += gridDim.x / ctas) {
        const int64_t at = row * cols;
        const T* hr = static_cast<const T*>(p.h) + at;
        const T* ar = static_cast<const T*>(p.a) + at;
        const T* dyr = static_cast<const T*>(p.dy) + at;
        const bool has_dh = p.dh != nullptr;
        const T* dhr = has_dh ? static_cast<const T*>(p.dh) + at : dyr;  // (without dh there is dy, and no branch)
        const ReadParam gate(p.gate ? p.gate + row / p.group_rows * cols : nullptr, 1);
        auto u_of = [&](int c) { return to_float(dyr[c]) * pre_w(c); };
        // squares of h and a, u h, u, h and a, about shifts
        float kh = LAYER && PRE ? lane_mean(to_float(hr[start])) : 0.0f;
        float ka = LAYER && POST ? lane_mean(to_float(ar[start])) : 0.0f;
        float s[6], off_h, off_a, sq_h, sq_a;
        for (bool again = false;; again = true) {
            rr.sums<6>([&](int c) {
                const float h = PRE ? to_float(hr[c]) - kh : 0.0f, a = POST ? to_float(ar[c]) - ka : 0.0f;
                const float u = PRE ? u_of(c) : 0.0f;
                return Values<6>{{h * h, a * a, u * h, LAYER ? u : 0.0f, LAYER ? h : 0.0f, LAYER ? a : 0.0f}};
            }, s);
            off_h = s[4] * inv_n;
            off_a = s[5] * inv_n;
            sq_h = s[0];
            sq_a = s[1];
            if (!LAYER) break;
            bool far_h, far_a;
            sq_h = squares_about_mean(s[0], s[4], off_h, far_h);
            sq_a = squares_about_mean(s[1], s[5], off_a, far_a);
            if (again || (!far_h && !far_a)) break;  // (alike in all threads of the row)
            kh += off_h;
            ka += off_a;
        }
        const float mh = kh + off_h, ma = ka + off_a, c1 = s[3] * inv_n;
        const float rh = PRE ? rsqrtf(fmaf(sq_h, inv_n, p.eps)) : 0.0f;
        const float ra = POST ? rsqrtf(fmaf(sq_a, inv_n, p.eps)) : 0.0f;
        const float c2 = fmaf(-off_h, s[3], s[2]) * inv_n * rh;
        auto ah_of = [&](int c) { return POST ? (to_float(ar[c]) - ma) * ra : 0.0f; };
        auto d_of = [&](int c) {
            const float v = to_float(dhr[c]);
            const float d = has_dh ? v : 0.0f;
            return PRE ? d + rh * (u_of(c) - c1 - (to_float(hr[c]) - mh) * rh * c2) : d;
        };
        auto q_of = [&](float d, int c) { return p.bs * d * gate(c) * (POST ? post_w(c) : 1.0f); };
        float e[2] = {0.0f, 0.0f};
        if (POST) {
            rr.sums<2>([&](int c) {
                const float q = q_of(d_of(c), c);
                return Values<2>{{LAYER ? q : 0.0f, q * ah_of(c)}};
            }, e);
            e[0] *= inv_n;
            e[1] *= inv_n;
        }
        if (p.sums && threadIdx.x == 0 && rr.begin == 0) {
            float* st = p.stats + row * kBlockStats;
            st[0] = mh;
            st[1] = rh;
            st[2] = c1;
            st[3] = c2;
            st[4] = ma;
            st[5] = ra;
        }
        rr.columns(
            [&](int c) {
                const float d = d_of(c);
                const float q = q_of(d, c);
                return Values<2>{{p.rs * d, POST ? ra * (q - e[0] - ah_of(c) * e[1]) : q}};
            },
            [&](int c, const Values<2>& v) {
                static_cast<T*>(p.dx)[at + c] = from_float<T>(v.v[0]);
                static_cast<T*>(p.da)[at + c] = from_float<T>(v.v[1]);
            });
    }
    if (ctas > 1) cg::this_cluster().sync();  // no CTA leaves while another may still write to it
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

// A CTA of 512 threads takes TILE columns, 512 / TILE slabs at a time (TILE 8, one sector, for short rows, whose
// columns are few and slabs many). The partials come from L2 and latency is all there is: 16 loads a thread are
// under way at once, two CTAs fit an SM, and the threads of a column meet twice, not in a tree of barriers.
constexpr int kFinishThreads = 512;

// v[i] += a column's sum of vector first_vector + stride i of slabs first, first + step, ... < end.
template <int N>
__device__ __forceinline__ void slab_sums(const float* part, int cols, int vectors, int first_vector, int stride, int first,
                                          int end, int step, float (&v)[N]) {
    constexpr int U = 16 / N;
    const int64_t slab_floats = static_cast<int64_t>(vectors) * cols, vector_floats = static_cast<int64_t>(stride) * cols;
    for (int s = first; s < end; s += U * step) {
        const float* q0 = part + s * slab_floats + static_cast<int64_t>(first_vector) * cols;
        float q[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < N; ++i) q[u][i] = s + u * step < end ? q0[u * step * slab_floats + i * vector_floats] : 0.0f;
#pragma unroll
        for (int o = U / 2; o >= 1; o /= 2)
#pragma unroll
            for (int u = 0; u < o; ++u)
#pragma unroll
                for (int i = 0; i < N; ++i) q[u][i] += q[u + o][i];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += q[0][i];
    }
}

template <bool LAYER, int TILE>
__global__ void __launch_bounds__(kFinishThreads, 2) bwd_finish_kernel(const BlockBwArgs p) {
    constexpr int V = LAYER ? 4 : 2;
    constexpr int H = V / 2;  // vectors of a norm: dy hh, dy (pre); D ah, D (post)
    constexpr int SUBS = kFinishThreads / TILE;
    constexpr int PAD = TILE + 1;
    __shared__ float red[V][SUBS * PAD];
    __shared__ float sum[V][TILE];
    const int tid = static_cast<int>(threadIdx.x), lane = tid % TILE, sub = tid / TILE;
    const int cols = p.cols;
    const int c = static_cast<int>(blockIdx.x) * TILE + lane;
    const bool ok = c < cols;
    const float* part = p.part + (ok ? c : 0);
    // (inputs, not results of the kernel before: they may be read while it ends)
    const float ow = ok && p.post && p.post_w ? __ldg(p.post_w + c) : 1.0f;
    const float ob = ok && p.post && p.post_b ? __ldg(p.post_b + c) : 0.0f;
    const bool need_a = p.post || p.dgate;
    const bool single = p.groups == 1;              // one gate row: its sums are the columns' own
    const bool grouped = p.slices > 0 && !single;  // several gate rows of several slabs each
    const float g0 = ok && p.gate && single ? __ldg(p.gate + c) : 1.0f;
    pdl_enter();

    float pre[H] = {}, post[H] = {};
    const int slabs = static_cast<int>(p.slabs), slices = static_cast<int>(p.slices);
    if (p.pre && need_a && !grouped) {
        float all[V] = {};
        slab_sums<V>(part, cols, V, 0, 1, sub, slabs, SUBS, all);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            pre[i] = all[2 * i];
            post[i] = all[2 * i + 1];
        }
    } else {
        if (p.pre) slab_sums<H>(part, cols, V, 0, 2, sub, slabs, SUBS, pre);
        if (need_a && !grouped) slab_sums<H>(part, cols, V, 1, 2, sub, slabs, SUBS, post);
    }
    if (need_a && grouped) {
        // `per` (a power of two) threads of a column to each gate row
        int per = SUBS;
        while (per > 1 && SUBS / per < p.groups) per >>= 1;
        const int member = sub & (per - 1);
        for (int64_t g = sub / per; g < p.groups; g += SUBS / per) {
            float t[H] = {};
            slab_sums<H>(part, cols, V, 1, 2, static_cast<int>(g) * slices + member, static_cast<int>(g + 1) * slices, per, t);
            if (per > 1) {  // (then there is one round: the threads without a gate row come with zeros below)
#pragma unroll
                for (int i = 0; i < H; ++i) post[i] = t[i];
                break;
            }
            const float b = H > 1 ? t[H - 1] : 0.0f;
            if (ok && p.dgate) p.dgate[g * cols + c] = p.bs * (ow * t[0] + ob * b);
            const float gate = ok ? p.gate[g * cols + c] : 0.0f;
#pragma unroll
            for (int i = 0; i < H; ++i) post[i] = fmaf(gate, t[i], post[i]);
        }
        if (per > 1) {
#pragma unroll
            for (int i = 0; i < H; ++i) red[i][sub * PAD + lane] = post[i];
            __syncthreads();
            const int64_t g = sub / per;
#pragma unroll
            for (int i = 0; i < H; ++i) post[i] = 0.0f;
            if (member == 0 && g < p.groups) {
#pragma unroll
                for (int i = 0; i < H; ++i)
                    for (int k = 0; k < per; ++k) post[i] += red[i][(sub + k) * PAD + lane];
                const float b = H > 1 ? post[H - 1] : 0.0f;
                if (ok && p.dgate) p.dgate[g * cols + c] = p.bs * (ow * post[0] + ob * b);
                const float gate = ok ? p.gate[g * cols + c] : 0.0f;
#pragma unroll
                for (int i = 0; i < H; ++i) post[i] *= gate;
            }
            __syncthreads();
        }
    }
    // over the threads of a column: a warp to each column and vector
#pragma unroll
    for (int i = 0; i < H; ++i) {
        red[i][sub * PAD + lane] = pre[i];
        red[H + i][sub * PAD + lane] = post[i];
    }
    __syncthreads();
#pragma unroll
    for (int q = tid / 32; q < V * TILE; q += kFinishThreads / 32) {
        const float* r = red[q / TILE] + q % TILE;
        float t = 0.0f;
#pragma unroll
        for (int k = tid % 32; k < SUBS; k += 32) t += r[k * PAD];
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(kFull, t, o);
        if (tid % 32 == 0) sum[q / TILE][q % TILE] = t;
    }
    __syncthreads();
    if (sub != 0 || !ok) return;
    if (p.pre && p.dpre_w) p.dpre_w[c] = sum[0][lane];
    const float a = sum[H][lane];
    if (p.post && p.dpost_w) p.dpost_w[c] = p.bs * (single ? g0 * a : a);
    if constexpr (LAYER) {
        if (p.pre && p.dpre_b) p.dpre_b[c] = sum[1][lane];
        if (p.post && p.dpost_b) p.dpost_b[c] = p.bs * (single ? g0 * sum[V - 1][lane] : sum[V - 1][lane]);
    }
    if (single && p.dgate) p.dgate[c] = p.bs * (ow * a + (LAYER ? ob * sum[V - 1][lane] : 0.0f));
}

template <class T, bool LAYER>
cudaError_t bwd_launch(const BlockBwArgs& in, cudaStream_t stream) {
    BlockBwArgs a = in;
    const unsigned tiles = static_cast<unsigned>((a.cols + kTile - 1) / kTile);
    // as many slabs as the column tiles leave of about 16 CTAs an SM
    block_slabs(&a, std::min<int64_t>(block_slab_limit(a.rows, a.cols), std::max(1u, 16 * 152 / tiles)));
    const int ctas = read_cluster(a.rows, a.cols);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.rows, 1 << 20)) * ctas;
    const auto kernel = a.pre && a.post ? bwd_read_kernel<T, LAYER, true, true>
                        : a.pre         ? bwd_read_kernel<T, LAYER, true, false>
                                        : bwd_read_kernel<T, LAYER, false, true>;
    cudaError_t e = launch_dependent(kernel, dim3(grid), kReadThreads, 0, ctas, stream, a);
    if (e != cudaSuccess || !a.sums) return e;
    e = launch_dependent(bwd_columns_kernel<T, LAYER>, dim3(tiles, static_cast<unsigned>(a.slabs)), kTile * 8, 0, 1, stream, a);
    if (e != cudaSuccess) return e;
    return launch_block_finish(LAYER ? TR_NORM_LAYER : TR_NORM_RMS, a, stream);
}

template <class T>
cudaError_t bwd_read(int kind, const BlockBwArgs& a, cudaStream_t stream) {
    return kind == TR_NORM_LAYER ? bwd_launch<T, true>(a, stream) : bwd_launch<T, false>(a, stream);
}

}  // namespace block

template <bool LAYER>
static cudaError_t finish(const BlockBwArgs& a, cudaStream_t stream) {
    using block::bwd_finish_kernel;
    using block::kFinishThreads;
    auto go = [&](auto kernel, int tile) {
        return launch_dependent(kernel, dim3(static_cast<unsigned>((a.cols + tile - 1) / tile)), kFinishThreads, 0, 1, stream, a);
    };
    // the widest tile that still makes a CTA for each of 152 SMs
    if (a.cols >= 32 * 152) return go(bwd_finish_kernel<LAYER, 32>, 32);
    if (a.cols >= 16 * 152) return go(bwd_finish_kernel<LAYER, 16>, 16);
    return go(bwd_finish_kernel<LAYER, 8>, 8);
}

cudaError_t launch_block_finish(int kind, const BlockBwArgs& a, cudaStream_t stream) {
    return kind == TR_NORM_LAYER ? finish<true>(a, stream) : finish<false>(a, stream);
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
