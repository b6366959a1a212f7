// The gated residual norm's backward with the rows on chip (see k_block_bwd.cu for
// the formulas).
//
// HBM-bound: h, a, dy and dh are read and dx and da written once. A thread owns the same columns of
// every row of its slab, so the column sums stay in its registers (32-bit) until the slab ends.
//
// With 16-bit types the work per byte is what limits: at 4096 columns a SM has 2090 cycles to
// the row. So the arithmetic is on pairs (f32x2), which norms there are is known when the kernel is
// compiled, and there is one exchange between warps a row: the next row's statistics travel with
// this row's sum of q ah. LayerNorm's squares are taken about the warp's own mean and moved to the
// row's when the warps meet (Chan, Golub and LeVeque 1979), so it needs no second exchange.
#pragma once

#include "tr_block_rows.cuh"

namespace tr {
namespace block {

// MODE: the norms there are, a mask of TR_BLOCK_POST and TR_BLOCK_PRE; 0: as p says.
template <class T, bool LAYER, int S, bool ODD, bool CLUSTER, int MODE, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) bwd_kernel(const BlockBwArgs p, const RowShape g) {
    constexpr int E = 16 / static_cast<int>(sizeof(T));
    constexpr int P = E / 2;       // pairs of a slot
    constexpr int K = S * P;       // pairs of a thread
    constexpr int V = LAYER ? 4 : 2;
    const bool pre = MODE ? (MODE & TR_BLOCK_PRE) != 0 : p.pre != 0;
    const bool post = MODE ? (MODE & TR_BLOCK_POST) != 0 : p.post != 0;
    extern __shared__ uint4 smem[];
    const int tt = g.warps * 32;  // a team's threads in this CTA
    const int team = CLUSTER ? 0 : static_cast<int>(threadIdx.x) / tt;
    const int t = static_cast<int>(threadIdx.x) - team * tt;
    const int rank = CLUSTER ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
    const int cols = p.cols;
    const int col0 = rank * g.cta_vecs * E;  // this CTA's first column
    const Lanes<T, S, ODD> ln(t, tt, cols, col0, g.cta_vecs);
    const float inv_n = 1.0f / static_cast<float>(cols);
    Exchange<CLUSTER, 4> ex{reinterpret_cast<float*>(smem) + team * (team_bytes(g) / 4), g.warps * g.cluster,
                            rank * g.warps + (t >> 5), team, g.warps};
    const int stage_bytes = g.tensors * g.tensor_bytes;
    char* ring = reinterpret_cast<char*>(smem) + fixed_bytes(g) + team * g.stages * stage_bytes;
    if constexpr (LAYER) ex.template count_columns<S, E, ODD>(cols, g.cta_vecs, t);
    if constexpr (CLUSTER) cg::this_cluster().sync();  // every CTA of the cluster runs before it is written to
    pdl_enter();

    const int64_t index = CLUSTER ? blockIdx.x / g.cluster : static_cast<int64_t>(blockIdx.x) * g.teams + team;
    if (index >= p.slabs) return;  // (a whole cluster, or a whole team)
    const SlabRows slab = slab_rows(p, index);

    // ---- the ring: h and dy (pre), a, dh, each where there is one ----
    const bool need_a = post || p.dgate;
    const int at_dy = pre ? g.tensor_bytes : 0;
    const int at_a = pre ? 2 * g.tensor_bytes : 0;
    const int at_dh = at_a + (need_a ? g.tensor_bytes : 0);
    auto fetch = [&](int64_t row, int stage) {
        if (row < slab.end) {
            char* to = ring + stage * stage_bytes;
            if (pre) {
                ln.fetch(p.h, p.rows, row, to);
                ln.fetch(p.dy, p.rows, row, to + at_dy);
            }
            if (need_a) ln.fetch(p.a, p.rows, row, to + at_a);
            if (p.dh) ln.fetch(p.dh, p.rows, row, to + at_dh);
        }
        cp_async_commit();
    };
    auto at0 = [&](const float* w) { return w ? w + col0 : nullptr; };

    // the slab's column sums dy hh and dy; those of the running gate row, D ah and D
    float2 sum0[K], sumA[K], sum1[LAYER ? K : 1], sumB[LAYER ? K : 1];
    float2 w[K], qw[K];  // the pre-norm's weight; bs gate w_post
#pragma unroll
    for (int k = 0; k < K; ++k) {
        sum0[k] = sumA[k] = both(0.0f);
        if constexpr (LAYER) sum1[k] = sumB[k] = both(0.0f);
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        float2 v[P];
        ln.param(pre ? at0(p.pre_w) : nullptr, s, 1.0f, v);
#pragma unroll
        for (int j = 0; j < P; ++j) w[s * P + j] = v[j];
    }
    auto gate_row = [&](int64_t row) { return p.gate ? p.gate + row / p.group_rows * cols + col0 : nullptr; };
    auto enter_group = [&](int64_t row) {
        const float* gr = gate_row(row);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float2 o[P], v[P];
            ln.param(post ? at0(p.post_w) : nullptr, s, 1.0f, o);
            ln.param(gr, s, 1.0f, v);
#pragma unroll
            for (int j = 0; j < P; ++j) qw[s * P + j] = __fmul2_rn(v[j], __fmul2_rn(both(p.bs), o[j]));
        }
    };
    // a whole group is done: its gate gradient is final, and its share of the post-norm's column
    // sums goes to the slab's partials, which no other thread touches
    bool flushed = false;
    auto leave_group = [&](int64_t row) {
        const float* gr = gate_row(row);
        float* dg = p.dgate ? p.dgate + row / p.group_rows * cols + col0 : nullptr;
        float* part = p.part + index * V * cols + col0;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float2 o[P], ob[P], gate[P];
            ln.param(post ? at0(p.post_w) : nullptr, s, 1.0f, o);
            ln.param(post ? at0(p.post_b) : nullptr, s, 0.0f, ob);
            ln.param(gr, s, 1.0f, gate);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int k = s * P + j;
                auto one = [&](int c, float wt, float bias, float gt, float a, float b) {
                    if (dg) dg[c] = p.bs * (LAYER ? fmaf(wt, a, bias * b) : wt * a);
                    part[cols + c] = fmaf(gt, a, flushed ? part[cols + c] : 0.0f);
                    if constexpr (LAYER) part[3 * cols + c] = fmaf(gt, b, flushed ? part[3 * cols + c] : 0.0f);
                };
                const float2 b = LAYER ? sumB[LAYER ? k : 0] : both(0.0f);
                if (ln.in(s, 2 * j)) one(ln.column(s, 2 * j), o[j].x, ob[j].x, gate[j].x, sumA[k].x, b.x);
                if (ln.in(s, 2 * j + 1)) one(ln.column(s, 2 * j + 1), o[j].y, ob[j].y, gate[j].y, sumA[k].y, b.y);
                sumA[k] = both(0.0f);
                if constexpr (LAYER) sumB[k] = both(0.0f);
            }
        }
        flushed = true;
    };
    auto about = [&](float2 v, float m, bool x_in, bool y_in) {  // v - m; 0 outside the row
        if constexpr (!LAYER) return v;
        float2 c = __fadd2_rn(v, both(-m));
        if (!x_in) c.x = 0.0f;
        if (!y_in) c.y = 0.0f;
        return c;
    };

    // ---- a row's statistics ----
    float mean_h = 0.0f, mean_a = 0.0f, c1 = 0.0f;  // LayerNorm: means of h, a, u
    // LayerNorm: the thread's sums of h, a and u
    auto plain_sums = [&](const char* m, int64_t row, float (&v)[4]) {
        float2 h2 = both(0.0f), a2 = both(0.0f), u2 = both(0.0f);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float2 x[P], y[P];
            if (pre) {
                ln.load(m, p.h, row, s, x);
                ln.load(m + at_dy, p.dy, row, s, y);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    h2 = __fadd2_rn(h2, x[j]);
                    u2 = __ffma2_rn(y[j], w[s * P + j], u2);
                }
            }
            if (post) {
                ln.load(m + at_a, p.a, row, s, x);
#pragma unroll
                for (int j = 0; j < P; ++j) a2 = __fadd2_rn(a2, x[j]);
            }
        }
        v[0] = h2.x + h2.y;
        v[1] = a2.x + a2.y;
        v[2] = u2.x + u2.y;
    };
    // the thread's sums of (h - mh)^2, (a - ma)^2 and u (h - mh)
    auto square_sums = [&](const char* m, int64_t row, float mh, float ma, float (&v)[4]) {
        float2 h2 = both(0.0f), a2 = both(0.0f), u2 = both(0.0f);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float2 x[P], y[P];
            if (pre) {
                ln.load(m, p.h, row, s, x);
                ln.load(m + at_dy, p.dy, row, s, y);
                ln.pairs(s, [&](int j, bool xi, bool yi) {
                    const float2 c = about(x[j], mh, xi, yi);
                    h2 = __ffma2_rn(c, c, h2);
                    u2 = __ffma2_rn(__fmul2_rn(y[j], w[s * P + j]), c, u2);
                });
            }
            if (post) {
                ln.load(m + at_a, p.a, row, s, x);
                ln.pairs(s, [&](int j, bool xi, bool yi) {
                    const float2 c = about(x[j], ma, xi, yi);
                    a2 = __ffma2_rn(c, c, a2);
                });
            }
        }
        v[0] = h2.x + h2.y;
        v[1] = a2.x + a2.y;
        v[2] = u2.x + u2.y;
    };
    // The statistics of row `row` staged at m (none when it is not there: `more` is false), with the sums of q
    // and q (a - mean) of the row before, which end in qs and qa. D = dh + r_h (u - c1 - (h - mean) k2) with
    // k2 = r_h^2 mean(u (h - mean)). rsqrtf is good to 2^-22, as the sums are.
    float rh = 0.0f, ra = 0.0f, k2 = 0.0f;
    auto statistics = [&](const char* m, int64_t row, bool more, float& qs, float& qa, auto&& between) {
        [[maybe_unused]] float v[4] = {0.0f, 0.0f, 0.0f, qs};
        float w4[4] = {0.0f, 0.0f, 0.0f, qa};
        if constexpr (LAYER) {
            if (more) plain_sums(m, row, v);
            ex.template moments<2>(
                v, w4, inv_n,
                [&](const float (&mean)[2], float (&o)[4]) {
                    if (more) square_sums(m, row, mean[0], mean[1], o);
                },
                [](int i, float n, const float (&d)[2], const float (&sum)[4]) {
                    return i < 2 ? n * d[i < 2 ? i : 0] * d[i < 2 ? i : 0] : i == 2 ? d[0] * sum[2] : 0.0f;
                });
            qs = v[3];
        } else {
            if (more) square_sums(m, row, 0.0f, 0.0f, w4);
            ex.sums(w4);
        }
        qa = w4[3];
        between();
        if constexpr (LAYER) {
            mean_h = v[0] * inv_n;
            mean_a = v[1] * inv_n;
            c1 = v[2] * inv_n;
        }
        if (pre) {
            rh = rsqrtf(fmaf(w4[0], inv_n, p.eps));
            k2 = w4[2] * inv_n * rh * rh;
        }
        if (post) ra = rsqrtf(fmaf(w4[1], inv_n, p.eps));
    };

    // ---- the first row ----
    auto odd_barrier = [&]() {
        if constexpr (CLUSTER) __syncthreads();
        else team_barrier(team, g.warps);
    };
    for (int i = 0; i + 1 < g.stages; ++i) fetch(slab.begin + i, i);
    ring_wait(g.stages, 2);
    if constexpr (ODD) odd_barrier();
    {
        float qs = 0.0f, qa = 0.0f;
        statistics(ring, slab.begin, true, qs, qa, [] {});
    }

    int stage = 0, fill = g.stages - 1;
    int64_t left = 0;  // rows of the running group still to come
    for (int64_t row = slab.begin; row < slab.end; ++row) {
        if (left == 0) {
            enter_group(row);
            left = p.slices > 0 ? slab.end - slab.begin : p.group_rows;
        }
        if constexpr (ODD) {  // the next row is here, and every thread is done with the row before
            ring_wait(g.stages, 1);
            odd_barrier();
        }
        fetch(row + g.stages - 1, fill);
        fill = fill + 1 == g.stages ? 0 : fill + 1;
        const char* m = ring + stage * stage_bytes;
        stage = stage + 1 == g.stages ? 0 : stage + 1;
        const char* next = ring + stage * stage_bytes;

        // D, dx, the column sums of the pre-norm, and the sums of q (a - mean) and q
        float2 d[K], av[K];
        float2 qa2 = both(0.0f), qs2 = both(0.0f);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float2 x[P], y[P], o[P];
            if (p.dh) {
                ln.load(m + at_dh, p.dh, row, s, o);
            } else {
#pragma unroll
                for (int j = 0; j < P; ++j) o[j] = both(0.0f);
            }
            if (pre) {
                ln.load(m, p.h, row, s, x);
                ln.load(m + at_dy, p.dy, row, s, y);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const int k = s * P + j;
                    const float2 c = LAYER ? __fadd2_rn(x[j], both(-mean_h)) : x[j];
                    sum0[k] = __ffma2_rn(__fmul2_rn(y[j], both(rh)), c, sum0[k]);
                    if constexpr (LAYER) sum1[k] = __fadd2_rn(sum1[k], y[j]);
                    const float2 u = LAYER ? __ffma2_rn(y[j], w[k], both(-c1)) : __fmul2_rn(y[j], w[k]);
                    o[j] = __ffma2_rn(both(rh), __ffma2_rn(c, both(-k2), u), o[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < P; ++j) {
                d[s * P + j] = o[j];
                o[j] = __fmul2_rn(o[j], both(p.rs));
            }
            ln.store(p.dx, row, s, o);
            if (need_a) {
                ln.load(m + at_a, p.a, row, s, x);
#pragma unroll
                for (int j = 0; j < P; ++j) av[s * P + j] = LAYER && post ? __fadd2_rn(x[j], both(-mean_a)) : x[j];
                if (post)
                    ln.pairs(s, [&](int j, bool xi, bool yi) {
                        float2 q = __fmul2_rn(d[s * P + j], qw[s * P + j]);
                        if (!xi) q.x = 0.0f;
                        if (!yi) q.y = 0.0f;
                        qa2 = __ffma2_rn(q, av[s * P + j], qa2);
                        if constexpr (LAYER) qs2 = __fadd2_rn(qs2, q);
                    });
            }
        }
        // the next row's statistics travel with this row's sums
        if constexpr (!ODD) ring_wait(g.stages, 2);
        float qs = qs2.x + qs2.y, qa = qa2.x + qa2.y;
        statistics(next, row + 1, row + 1 < slab.end, qs, qa, [&] {
            // da, and the column sums of the post-norm and the gate
            const float e1 = qs * inv_n, e2 = qa * inv_n * ra * ra;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float2 o[P];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const int k = s * P + j;
                    float2 q = __fmul2_rn(d[k], qw[k]);
                    if (need_a) {
                        float2 ah = av[k];
                        if (post) {
                            q = __ffma2_rn(av[k], both(-e2), q);
                            if constexpr (LAYER) q = __fadd2_rn(q, both(-e1));
                            q = __fmul2_rn(q, both(ra));
                            ah = __fmul2_rn(av[k], both(ra));
                        }
                        sumA[k] = __ffma2_rn(d[k], ah, sumA[k]);
                        if constexpr (LAYER) sumB[k] = __fadd2_rn(sumB[k], d[k]);
                    }
                    o[j] = q;
                }
                ln.store(p.da, row, s, o);
            }
            if (--left == 0 && p.slices == 0 && p.sums) leave_group(row);
        });
    }
    if (p.sums) {
        float* part = p.part + index * V * cols + col0;
        auto one = [&](int c, float a0, float a1, float b0, float b1) {
            part[c] = a0;
            if (p.slices > 0) part[cols + c] = a1;
            if constexpr (LAYER) {
                part[2 * cols + c] = b0;
                if (p.slices > 0) part[3 * cols + c] = b1;
            }
        };
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int k = s * P + j, l = LAYER ? k : 0;
                const float2 b0 = LAYER ? sum1[l] : both(0.0f), b1 = LAYER ? sumB[l] : both(0.0f);
                if (ln.in(s, 2 * j)) one(ln.column(s, 2 * j), sum0[k].x, sumA[k].x, b0.x, b1.x);
                if (ln.in(s, 2 * j + 1)) one(ln.column(s, 2 * j + 1), sum0[k].y, sumA[k].y, b0.y, b1.y);
            }
    }
    if constexpr (CLUSTER) cg::this_cluster().sync();  // no CTA leaves while another may still write to it
}

// ---- host side -------------------------------------------------------------

template <class T, bool LAYER, int S, bool ODD, bool CLUSTER, int MODE, int THREADS, int CTAS>
cudaError_t bwd_go(const BlockBwArgs& in, const RowShape& g, cudaStream_t stream) {
    BlockBwArgs a = in;
    const int threads = g.teams * g.warps * 32;
    const size_t smem = row_smem(g);
    const auto kernel = bwd_kernel<T, LAYER, S, ODD, CLUSTER, MODE, THREADS, CTAS>;
    const int64_t ctas = resident_ctas(reinterpret_cast<const void*>(kernel), threads, smem, g.cluster);
    if (ctas < 1) return cudaErrorInvalidConfiguration;
    block_slabs(&a, std::min(ctas * g.teams / g.cluster, block_slab_limit(a.rows, a.cols)));
    const unsigned grid = static_cast<unsigned>((a.slabs + g.teams - 1) / g.teams * g.cluster);
    cudaError_t e = launch_dependent(kernel, dim3(grid), threads, smem, g.cluster, stream, a, g);
    if (e != cudaSuccess || !a.sums) return e;
    return launch_block_finish(LAYER ? TR_NORM_LAYER : TR_NORM_RMS, a, stream);
}

// Aligned rows of one CTA are compiled for each pair of norms, and for CTAs of at most 320 threads
// with registers for two an SM.
template <class T, bool LAYER, int S, int MODE>
cudaError_t bwd_aligned(const BlockBwArgs& a, const RowShape& g, cudaStream_t stream) {
    if constexpr (S == 1) {
        if (g.teams * g.warps <= 10) return bwd_go<T, LAYER, S, false, false, MODE, 320, 2>(a, g, stream);
    }
    return bwd_go<T, LAYER, S, false, false, MODE, 512, 1>(a, g, stream);
}

template <class T, bool LAYER, int S>
cudaError_t bwd_slots(bool odd, const BlockBwArgs& a, const RowShape& g, cudaStream_t stream) {
    if (g.cluster > 1)
        return odd ? bwd_go<T, LAYER, S, true, true, 0, 512, 1>(a, g, stream) : bwd_go<T, LAYER, S, false, true, 0, 512, 1>(a, g, stream);
    if (odd) return bwd_go<T, LAYER, S, true, false, 0, 512, 1>(a, g, stream);
    if (a.pre && a.post) return bwd_aligned<T, LAYER, S, TR_BLOCK_PRE | TR_BLOCK_POST>(a, g, stream);
    return a.pre ? bwd_aligned<T, LAYER, S, TR_BLOCK_PRE>(a, g, stream) : bwd_aligned<T, LAYER, S, TR_BLOCK_POST>(a, g, stream);
}

template <class T, bool LAYER>
cudaError_t bwd_kind(const BlockBwArgs& a, bool* done, cudaStream_t stream) {
    const int tensors = (a.pre ? 2 : 0) + (a.post || a.dgate ? 1 : 0) + (a.dh ? 1 : 0);
    const bool odd = !rows_aligned(static_cast<int64_t>(a.cols) * static_cast<int>(sizeof(T)),
                                   {a.pre ? a.h : nullptr, a.pre ? a.dy : nullptr, a.post || a.dgate ? a.a : nullptr, a.dh, a.dx, a.da});
    int slots = 0;
    const RowShape g = row_shape<T>(a.cols, tensors, odd, 1, &slots);
    *done = g.warps > 0;
    if (!*done) return cudaSuccess;
    if constexpr (sizeof(T) == 4) {
        if (slots == 2) return bwd_slots<T, LAYER, 2>(odd, a, g, stream);
    }
    return bwd_slots<T, LAYER, 1>(odd, a, g, stream);
}

}  // namespace block
}  // namespace tr
