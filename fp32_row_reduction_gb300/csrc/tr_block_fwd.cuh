// The gated residual norm with the rows on chip: h = rs x + bs gate post(a), y = pre(h).
//
// HBM-bound: x and a are read, h and y written once. A row's y waits for the statistics of h, which
// wait for those of a; so that a row costs one exchange between its warps, the sum over h of a row
// travels with the sum over a of the next one. The parameters of a thread's columns stay in its
// registers for all its rows.
#pragma once

#include "tr_block_rows.cuh"

namespace tr {
namespace block {

template <class T, bool LAYER, int S, bool ODD, bool CLUSTER>
__global__ void __launch_bounds__(512, 2) fwd_kernel(const BlockArgs p, const RowShape g, const int64_t slabs) {
    constexpr int E = 16 / static_cast<int>(sizeof(T));
    constexpr int P = E / 2;  // pairs of a slot
    constexpr int K = S * P;  // pairs of a thread
    extern __shared__ uint4 smem[];
    const int tt = g.warps * 32;  // a team's threads in this CTA
    const int team = CLUSTER ? 0 : static_cast<int>(threadIdx.x) / tt;
    const int t = static_cast<int>(threadIdx.x) - team * tt;
    const int rank = CLUSTER ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
    const int cols = p.cols;
    const int col0 = rank * g.cta_vecs * E;  // this CTA's first column
    const Lanes<T, S, ODD> ln(t, tt, cols, col0, g.cta_vecs);
    const float inv_n = 1.0f / static_cast<float>(cols);
    Exchange<CLUSTER, 2> ex{reinterpret_cast<float*>(smem) + team * (team_bytes(g) / 4), g.warps * g.cluster,
                            rank * g.warps + (t >> 5), team, g.warps};
    const int stage_bytes = g.tensors * g.tensor_bytes;
    char* ring = reinterpret_cast<char*>(smem) + fixed_bytes(g) + team * g.stages * stage_bytes;
    if constexpr (LAYER) ex.template count_columns<S, E, ODD>(cols, g.cta_vecs, t);
    if constexpr (CLUSTER) cg::this_cluster().sync();  // every CTA of the cluster runs before it is written to
    pdl_enter();

    const int64_t index = CLUSTER ? blockIdx.x / g.cluster : static_cast<int64_t>(blockIdx.x) * g.teams + team;
    if (index >= slabs) return;  // (a whole team)
    const int64_t begin = p.rows * index / slabs, end = p.rows * (index + 1) / slabs;

    auto fetch = [&](int64_t row, int stage) {
        if (row < end) {
            char* to = ring + stage * stage_bytes;
            ln.fetch(p.a, p.rows, row, to);
            ln.fetch(p.x, p.rows, row, to + g.tensor_bytes);
        }
        cp_async_commit();
    };
    auto odd_barrier = [&]() {
        if constexpr (CLUSTER) __syncthreads();
        else team_barrier(team, g.warps);
    };
    for (int i = 0; i + 1 < g.stages; ++i) fetch(begin + i, i);

    auto at0 = [&](const float* w) { return w ? w + col0 : nullptr; };
    float2 gw[K], w[K];  // bs gate w_post;  the pre-norm's weight
#pragma unroll
    for (int s = 0; s < S; ++s) {
        float2 v[P];
        ln.param(at0(p.pre_w), s, 1.0f, v);
#pragma unroll
        for (int j = 0; j < P; ++j) w[s * P + j] = v[j];
    }
    auto gate_row = [&](int64_t row) { return p.gate ? p.gate + row / p.group_rows * cols + col0 : nullptr; };
    auto enter_group = [&](int64_t row) {
        const float* gr = gate_row(row);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float2 o[P], v[P];
            ln.param(at0(p.post_w), s, 1.0f, o);
            ln.param(gr, s, 1.0f, v);
#pragma unroll
            for (int j = 0; j < P; ++j) gw[s * P + j] = __fmul2_rn(v[j], __fmul2_rn(both(p.bs), o[j]));
        }
    };
    auto about = [&](float2 v, float m, bool x_in, bool y_in) {  // v - m; 0 outside the row
        if constexpr (!LAYER) return v;
        float2 c = __fadd2_rn(v, both(-m));
        if (!x_in) c.x = 0.0f;
        if (!y_in) c.y = 0.0f;
        return c;
    };

    float2 h[K];
    float ra = 1.0f, ma = 0.0f;  // of the row at work
    float rh = 1.0f, mh = 0.0f;
    // the sums over h (where `this_row`) and over a of row `row` staged at m (where `next_row`)
    auto statistics = [&](const char* m, int64_t row, bool this_row, bool next_row) {
        float q[2] = {0.0f, 0.0f};  // squares of h, of a
        auto squares = [&](float mean_h, float mean_a, float (&o)[2]) {
            float2 h2 = both(0.0f), a2 = both(0.0f);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if (p.pre && this_row)
                    ln.pairs(s, [&](int j, bool xi, bool yi) {
                        const float2 c = about(h[s * P + j], mean_h, xi, yi);
                        h2 = __ffma2_rn(c, c, h2);
                    });
                if (p.post && next_row) {
                    float2 x[P];
                    ln.load(m, p.a, row, s, x);
                    ln.pairs(s, [&](int j, bool xi, bool yi) {
                        const float2 c = about(x[j], mean_a, xi, yi);
                        a2 = __ffma2_rn(c, c, a2);
                    });
                }
            }
            o[0] = h2.x + h2.y;
            o[1] = a2.x + a2.y;
        };
        float v[2] = {0.0f, 0.0f};
        if constexpr (LAYER) {
            float2 h2 = both(0.0f), a2 = both(0.0f);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if (p.pre && this_row)
#pragma unroll
                    for (int j = 0; j < P; ++j) h2 = __fadd2_rn(h2, h[s * P + j]);
                if (p.post && next_row) {
                    float2 x[P];
                    ln.load(m, p.a, row, s, x);
#pragma unroll
                    for (int j = 0; j < P; ++j) a2 = __fadd2_rn(a2, x[j]);
                }
            }
            v[0] = h2.x + h2.y;
            v[1] = a2.x + a2.y;
            ex.template moments<2>(
                v, q, inv_n, [&](const float (&mean)[2], float (&o)[2]) { squares(mean[0], mean[1], o); },
                [](int i, float n, const float (&d)[2], const float (&)[2]) { return n * d[i] * d[i]; });
        } else {
            squares(0.0f, 0.0f, q);
            ex.sums(q);
        }
        // rsqrtf is good to 2^-22, as the sums are
        rh = rsqrtf(fmaf(q[0], inv_n, p.eps));
        if (p.post) ra = rsqrtf(fmaf(q[1], inv_n, p.eps));
        if constexpr (LAYER) {
            mh = v[0] * inv_n;
            if (p.post) ma = v[1] * inv_n;
        }
    };

    int64_t left = 0;  // rows of the running gate row still to come
    if (begin < end) {
        enter_group(begin);
        left = p.group_rows - begin % p.group_rows;
    }
    ring_wait(g.stages, 2);
    if constexpr (ODD) odd_barrier();
    if (p.post) statistics(ring, begin, false, begin < end);
    int stage = 0, fill = g.stages - 1;
    for (int64_t row = begin; row < end; ++row) {
        if (left == 0) {
            enter_group(row);
            left = p.group_rows;
        }
        --left;
        if constexpr (ODD) {  // the next row is here, and every thread is done with the row before
            ring_wait(g.stages, 1);
            odd_barrier();
        }
        fetch(row + g.stages - 1, fill);
        fill = fill + 1 == g.stages ? 0 : fill + 1;
        const char* m = ring + stage * stage_bytes;
        stage = stage + 1 == g.stages ? 0 : stage + 1;
        const char* next = ring + stage * stage_bytes;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float2 x[P], v[P];
            ln.load(m, p.a, row, s, v);
            ln.load(m + g.tensor_bytes, p.x, row, s, x);
            float2 b[LAYER ? P : 1], gt[LAYER ? P : 1];
            if constexpr (LAYER) {
                // bs gate b_post: read where there is a bias
                if (p.post_b) {
                    ln.param(at0(p.post_b), s, 0.0f, b);
                    ln.param(gate_row(row), s, 1.0f, gt);
#pragma unroll
                    for (int j = 0; j < P; ++j) x[j] = __ffma2_rn(both(p.rs), x[j], __fmul2_rn(__fmul2_rn(both(p.bs), gt[j]), b[j]));
                } else {
#pragma unroll
                    for (int j = 0; j < P; ++j) x[j] = __fmul2_rn(both(p.rs), x[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int k = s * P + j;
                const float2 c = LAYER ? __fadd2_rn(v[j], both(-ma)) : v[j];
                const float2 n = __fmul2_rn(c, both(ra));
                h[k] = LAYER ? __ffma2_rn(n, gw[k], x[j]) : __ffma2_rn(n, gw[k], __fmul2_rn(both(p.rs), x[j]));
                if constexpr (!ODD) {
                    if (!ln.in(s, 0)) h[k] = both(0.0f);
                } else {
                    if (!ln.in(s, 2 * j)) h[k].x = 0.0f;
                    if (!ln.in(s, 2 * j + 1)) h[k].y = 0.0f;
                }
                v[j] = h[k];
            }
            if (p.h) ln.store(p.h, row, s, v);
        }
        if constexpr (!ODD) ring_wait(g.stages, 2);
        statistics(next, row + 1, true, row + 1 < end);
        if (p.pre) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float2 o[P], b[P];
                if constexpr (LAYER) ln.param(at0(p.pre_b), s, 0.0f, b);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const int k = s * P + j;
                    const float2 c = LAYER ? __fadd2_rn(h[k], both(-mh)) : h[k];
                    const float2 n = __fmul2_rn(c, both(rh));
                    o[j] = LAYER ? __ffma2_rn(n, w[k], b[j]) : __fmul2_rn(n, w[k]);
                }
                ln.store(p.y, row, s, o);
            }
        }
    }
    if constexpr (CLUSTER) cg::this_cluster().sync();  // no CTA leaves while another may still write to it
}

// ---- host side -------------------------------------------------------------

template <class T, bool LAYER, int S, bool ODD, bool CLUSTER>
cudaError_t fwd_go(const BlockArgs& a, const RowShape& g, cudaStream_t stream) {
    const int threads = g.teams * g.warps * 32;
    const size_t smem = row_smem(g);
    const auto kernel = fwd_kernel<T, LAYER, S, ODD, CLUSTER>;
    const int64_t ctas = resident_ctas(reinterpret_cast<const void*>(kernel), threads, smem, g.cluster);
    if (ctas < 1) return cudaErrorInvalidConfiguration;
    const int64_t slabs = std::min(a.rows, ctas * g.teams / g.cluster);
    const unsigned grid = static_cast<unsigned>((slabs + g.teams - 1) / g.teams * g.cluster);
    return launch_dependent(kernel, dim3(grid), threads, smem, g.cluster, stream, a, g, slabs);
}

template <class T, bool LAYER, int S>
cudaError_t fwd_slots(bool odd, const BlockArgs& a, const RowShape& g, cudaStream_t stream) {
    if (g.cluster > 1) return odd ? fwd_go<T, LAYER, S, true, true>(a, g, stream) : fwd_go<T, LAYER, S, false, true>(a, g, stream);
    return odd ? fwd_go<T, LAYER, S, true, false>(a, g, stream) : fwd_go<T, LAYER, S, false, false>(a, g, stream);
}

template <class T, bool LAYER>
cudaError_t fwd_kind(const BlockArgs& a, bool* done, cudaStream_t stream) {
    const bool odd = !rows_aligned(static_cast<int64_t>(a.cols) * static_cast<int>(sizeof(T)), {a.x, a.a, a.h, a.y});
    int slots = 0;
    const RowShape g = row_shape<T>(a.cols, 2, odd, 2, &slots);
    *done = g.warps > 0;
    if (!*done) return cudaSuccess;
    if constexpr (sizeof(T) == 4) {
        if (slots == 2) return fwd_slots<T, LAYER, 2>(odd, a, g, stream);
    }
    return fwd_slots<T, LAYER, 1>(odd, a, g, stream);
}

}  // namespace block
}  // namespace tr
