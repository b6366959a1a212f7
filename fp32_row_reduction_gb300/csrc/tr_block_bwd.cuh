// The gated residual norm's backward with the rows on chip (see k_block_bwd.cu for
// the formulas).
//
// HBM-bound: h, a, dy and dh are read and dx and da written once (16384 x 4096 bf16, RMSNorm: 126 us, 6.4 TB/s, 94%
// of the measured copy rate). A thread owns the same columns of every row of its slab, so the column sums stay in its
// registers (32-bit) until the slab ends.
//
// With 16-bit types the work per byte is what limits: at 4096 columns a SM has 2090 cycles to
// the row. So the arithmetic is on pairs (f32x2), which norms there are is known when the kernel is
// compiled, and there is one exchange between warps a row: the next row's statistics travel with
// this row's sum of q ah. LayerNorm's sums are taken about a shift that each warp finds for itself
// (lane_mean), so means and variances need no second exchange and no second pass, but for a row whose shift is far
// from its mean (all rows far: 8192 x 4096 bf16 131 us against 96).
#pragma once

#include "tr_block_rows.cuh"

namespace tr {
namespace block {

// MODE: the norms there are, a mask of TR_BLOCK_POST and TR_BLOCK_PRE; 0: as p says.
template <class T, bool LAYER, int S, int LAYOUT, bool CLUSTER, int MODE, int THREADS, int CTAS, bool SPARAM>
__global__ void __launch_bounds__(THREADS, CTAS) bwd_kernel(const BlockBwArgs p, const RowShape g) {
    constexpr int E = 16 / static_cast<int>(sizeof(T));
    constexpr int P = E / 2;       // pairs of a slot
    constexpr int K = S * P;       // pairs of a thread
    constexpr int V = LAYER ? 4 : 2;
    constexpr bool ODD = LAYOUT == LAYOUT_ODD;
    constexpr bool RELOAD = SPARAM || (LAYER && S == 2);  // a - mean is taken from the ring again, not kept
    const bool pre = MODE ? (MODE & TR_BLOCK_PRE) != 0 : p.pre != 0;
    const bool post = MODE ? (MODE & TR_BLOCK_POST) != 0 : p.post != 0;
    extern __shared__ uint4 smem[];
    const int tt = g.warps * 32;  // a team's threads in this CTA
    const int team = CLUSTER ? 0 : static_cast<int>(threadIdx.x) / tt;
    const int t = static_cast<int>(threadIdx.x) - team * tt;
    const int rank = CLUSTER ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
    const int cols = p.cols;
    const int col0 = rank * g.cta_vecs * E;  // this CTA's first column
    const Lanes<T, S, LAYOUT> ln(t, tt, cols, col0, g.cta_vecs);
    const float inv_n = 1.0f / static_cast<float>(cols);
    char* const team_smem = reinterpret_cast<char*>(smem) + team * team_bytes(g);
    Exchange<CLUSTER, LAYER ? 8 : 4> ex(team_smem, g.warps * g.cluster, rank * g.warps + (t >> 5), team, g.warps, p.err, p.start);
    ex.init();
    const int stage_bytes = g.tensors * g.tensor_bytes;
    const RowStart<T, LAYOUT, CLUSTER> row_start(cols, ln.row_bytes);  // LayerNorm's
    char* starts = team_smem + exchange_bytes(g) + (t >> 5) * g.stages * g.sampled;
    char* ring = reinterpret_cast<char*>(smem) + fixed_bytes(g) + team * g.stages * stage_bytes;
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
            if constexpr (LAYER) {
                if (pre) row_start.fetch(p.h, row, starts + stage * g.sampled);
                if (post) row_start.fetch(p.a, row, starts + stage * g.sampled + kRowStartBytes);
            }
        }
        cp_async_commit();
    };
    auto at0 = [&](const float* w) { return w ? w + col0 : nullptr; };

    // the slab's column sums dy hh and dy; those of the running gate row, D ah and D
    float2 sum0[K], sumA[K], sum1[LAYER ? K : 1], sumB[LAYER ? K : 1];
    // the pre-norm's weight, and bs gate w_post: in registers, or (SPARAM) in the thread's own part of shared
    // memory, two pairs to a 16-byte word
    float2 w[SPARAM ? 1 : K], qw[SPARAM ? 1 : K];
    float4* own = reinterpret_cast<float4*>(team_smem + exchange_bytes(g) + g.warps * g.stages * g.sampled) + t;
    auto put_pairs = [&](int which, float2 (&reg)[SPARAM ? 1 : K], int s, const float2 (&v)[P]) {
#pragma unroll
        for (int j = 0; j < P; j += 2) {
            if constexpr (SPARAM) {
                own[(which * K + s * P + j) / 2 * tt] = make_float4(v[j].x, v[j].y, v[j + 1].x, v[j + 1].y);
            } else {
                reg[s * P + j] = v[j];
                reg[s * P + j + 1] = v[j + 1];
            }
        }
    };
    auto get_pairs = [&](int which, const float2 (&reg)[SPARAM ? 1 : K], int s, float2 (&v)[P]) {
#pragma unroll
        for (int j = 0; j < P; j += 2) {
            if constexpr (SPARAM) {
                const float4 q = own[(which * K + s * P + j) / 2 * tt];
                v[j] = make_float2(q.x, q.y);
                v[j + 1] = make_float2(q.z, q.w);
            } else {
                v[j] = reg[s * P + j];
                v[j + 1] = reg[s * P + j + 1];
            }
        }
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
        sum0[k] = sumA[k] = both(0.0f);
        if constexpr (LAYER) sum1[k] = sumB[k] = both(0.0f);
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        float2 v[P];
        ln.param(pre ? at0(p.pre_w) : nullptr, s, 1.0f, v);
        put_pairs(0, w, s, v);
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
            for (int j = 0; j < P; ++j) v[j] = __fmul2_rn(v[j], __fmul2_rn(both(p.bs), o[j]));
            put_pairs(1, qw, s, v);
        }
    };
    // a whole group is done: its gate gradient is final, and its share of the post-norm's column
    // sums goes to the slab's partials, which no other thread touches
    bool flushed = false;
    auto leave_group = [&](int64_t row) {
        const float* gr = gate_row(row);
        float* dg = p.dgate ? p.dgate + row / p.group_rows * cols + col0 : nullptr;
        float* part = p.part + index * V * cols + col0;
        // part += gate v
        auto add = [&](float* o, int s, const float2 (&gate)[P], const float2* v) {
            float2 x[P];
#pragma unroll
            for (int j = 0; j < P; ++j) x[j] = both(0.0f);
            if (flushed) ln.get_floats(o, s, x);
#pragma unroll
            for (int j = 0; j < P; ++j) x[j] = __ffma2_rn(gate[j], v[j], x[j]);
            ln.put_floats(o, s, x);
        };
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float2 o[P], gate[P];
            if (dg) {
                ln.param(post ? at0(p.post_w) : nullptr, s, p.bs, o);
                const float scale = post && p.post_w ? p.bs : 1.0f;
#pragma unroll
                for (int j = 0; j < P; ++j) o[j] = __fmul2_rn(__fmul2_rn(o[j], both(scale)), sumA[s * P + j]);
                if constexpr (LAYER) {
                    ln.param(post ? at0(p.post_b) : nullptr, s, 0.0f, gate);
#pragma unroll
                    for (int j = 0; j < P; ++j) o[j] = __ffma2_rn(__fmul2_rn(gate[j], both(p.bs)), sumB[LAYER ? s * P + j : 0], o[j]);
                }
                ln.put_floats(dg, s, o);
            }
            if (post) {
                ln.param(gr, s, 1.0f, gate);
                add(part + cols, s, gate, sumA + s * P);
                if constexpr (LAYER) add(part + 3 * cols, s, gate, sumB + s * P);
            }
#pragma unroll
            for (int j = 0; j < P; ++j) {
                sumA[s * P + j] = both(0.0f);
                if constexpr (LAYER) sumB[s * P + j] = both(0.0f);
            }
        }
        flushed = true;
    };
    // ---- a row's statistics ----
    float mean_h = 0.0f, mean_a = 0.0f, c1 = 0.0f;  // LayerNorm: means of h, a, u
    float rh = 0.0f, ra = 0.0f, k2 = 0.0f;
    bool far_h = false, far_a = false;  // LayerNorm: the row's sums are to be taken again
    // The statistics of row `row` in `stage` (when it is there: `more`), with the sums of q and q (a - mean) of the
    // row before, which end in qs and qa for between(). D = dh + r_h (u - c1 - (h - mean) k2) with
    // k2 = r_h^2 mean(u (h - mean)). rsqrtf is good to 2^-22, as the sums are.
    // Sums of row `row` staged at m about sh and sa: squares of h and a, and u h; sum[3] as it comes; for LayerNorm u,
    // h and a, and sum[7] as it comes.
    auto sums_about = [&](const char* m, int64_t row, bool more, float sh, float sa, float (&sum)[LAYER ? 8 : 4]) {
        float2 hh = both(0.0f), aa = both(0.0f), uh = both(0.0f), u1 = both(0.0f), h1 = both(0.0f), a1 = both(0.0f);
        if (more) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float2 x[P], y[P];
                auto shifted = [&](float2 v, float shift, bool xi, bool yi) {
                    if constexpr (!LAYER) return v;
                    float2 c = __fadd2_rn(v, both(-shift));
                    if (!xi) c.x = 0.0f;
                    if (!yi) c.y = 0.0f;
                    return c;
                };
                if (pre) {
                    ln.load(m, p.h, row, s, x);
                    ln.load(m + at_dy, p.dy, row, s, y);
                    float2 wv[P];
                    get_pairs(0, w, s, wv);
                    ln.pairs(s, [&](int j, bool xi, bool yi) {
                        const float2 c = shifted(x[j], sh, xi, yi);
                        const float2 u = __fmul2_rn(y[j], wv[j]);
                        hh = __ffma2_rn(c, c, hh);
                        uh = __ffma2_rn(u, c, uh);
                        if constexpr (LAYER) {
                            h1 = __fadd2_rn(h1, c);
                            u1 = __fadd2_rn(u1, u);
                        }
                    });
                }
                if (post) {
                    ln.load(m + at_a, p.a, row, s, x);
                    ln.pairs(s, [&](int j, bool xi, bool yi) {
                        const float2 c = shifted(x[j], sa, xi, yi);
                        aa = __ffma2_rn(c, c, aa);
                        if constexpr (LAYER) a1 = __fadd2_rn(a1, c);
                    });
                }
            }
        }
        sum[0] = hh.x + hh.y;
        sum[1] = aa.x + aa.y;
        sum[2] = uh.x + uh.y;
        if constexpr (LAYER) {
            sum[4] = u1.x + u1.y;
            sum[5] = h1.x + h1.y;
            sum[6] = a1.x + a1.y;
        }
        ex.sums(sum);
    };
    auto statistics = [&](int stage, int64_t row, bool more, float& qs, float& qa, auto&& between) {
        const char* m = ring + stage * stage_bytes;
        float sh = 0.0f, sa = 0.0f;
        if constexpr (LAYER) {
            __syncwarp();
            if (pre && more) sh = lane_mean(row_start.get(p.h, row, starts + stage * g.sampled, m));
            if (post && more) sa = lane_mean(row_start.get(p.a, row, starts + stage * g.sampled + kRowStartBytes, m + at_a));
        }
        float v[LAYER ? 8 : 4];
        v[3] = qa;
        if constexpr (LAYER) v[7] = qs;
        sums_about(m, row, more, sh, sa, v);
        qa = v[3];
        float sq_h = v[0], sq_a = v[1], sum_uh = v[2], next_h = 0.0f, next_a = 0.0f, next_c1 = 0.0f;
        if constexpr (LAYER) {
            qs = v[7];
            const float dh = v[5] * inv_n, da = v[6] * inv_n;  // the means, from the shifts
            sq_h = squares_about_mean(v[0], v[5], dh, far_h);
            sq_a = squares_about_mean(v[1], v[6], da, far_a);
            sum_uh = fmaf(-dh, v[4], v[2]);
            next_h = sh + dh;
            next_a = sa + da;
            next_c1 = v[4] * inv_n;
        }
        between();
        mean_h = next_h;
        mean_a = next_a;
        c1 = next_c1;
        if (pre) {
            rh = rsqrtf(fmaf(sq_h, inv_n, p.eps));
            k2 = sum_uh * inv_n * rh * rh;
        }
        if (post) ra = rsqrtf(fmaf(sq_a, inv_n, p.eps));
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
        statistics(0, slab.begin, true, qs, qa, [] {});
    }

    int stage = 0, fill = g.stages - 1;
    int64_t left = 0;  // rows of the running group still to come
    int64_t row = slab.begin;
    // Sums about a shift too far from the mean are taken again about that mean (by all warps of the row alike), before the
    // row uses them, between two rows. A test in the middle of a row's chain, where the sums come in, costs 8192 x 4096 f32
    // 47 us.
    auto take_again = [&]() {
        float v[LAYER ? 8 : 4] = {};
        sums_about(ring + stage * stage_bytes, row, true, mean_h, mean_a, v);
        if constexpr (LAYER) {
            const float dh = v[5] * inv_n, da = v[6] * inv_n;
            bool again;  // (not asked: the shift is the mean)
            if (far_h) {
                rh = rsqrtf(fmaf(squares_about_mean(v[0], v[5], dh, again), inv_n, p.eps));
                k2 = fmaf(-dh, v[4], v[2]) * inv_n * rh * rh;
                mean_h += dh;
            }
            if (far_a) {
                ra = rsqrtf(fmaf(squares_about_mean(v[1], v[6], da, again), inv_n, p.eps));
                mean_a += da;
            }
        }
        far_h = far_a = false;
    };
    auto one_row = [&]() {
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
        const bool more = row + 1 < slab.end;

        // D, dx, the column sums of the pre-norm, and the sums of q (a - mean) and q
        float2 d[K], av[RELOAD ? 1 : K];  // D, and a - mean
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
                float2 wv[P];
                get_pairs(0, w, s, wv);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const int k = s * P + j;
                    const float2 c = LAYER ? __fadd2_rn(x[j], both(-mean_h)) : x[j];
                    sum0[k] = __ffma2_rn(__fmul2_rn(y[j], both(rh)), c, sum0[k]);
                    if constexpr (LAYER) sum1[k] = __fadd2_rn(sum1[k], y[j]);
                    const float2 u = LAYER ? __ffma2_rn(y[j], wv[j], both(-c1)) : __fmul2_rn(y[j], wv[j]);
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
                for (int j = 0; j < P; ++j) {
                    if (LAYER && post) x[j] = __fadd2_rn(x[j], both(-mean_a));
                    if constexpr (!RELOAD) av[s * P + j] = x[j];
                }
                float2 qv[P];
                get_pairs(1, qw, s, qv);
                if (post)
                    ln.pairs(s, [&](int j, bool xi, bool yi) {
                        float2 q = __fmul2_rn(d[s * P + j], qv[j]);
                        if (!xi) q.x = 0.0f;
                        if (!yi) q.y = 0.0f;
                        qa2 = __ffma2_rn(q, x[j], qa2);
                        if constexpr (LAYER) qs2 = __fadd2_rn(qs2, q);
                    });
            }
        }
        // the next row's statistics travel with this row's sums
        if constexpr (!ODD) ring_wait(g.stages, 2);
        float qs = qs2.x + qs2.y, qa = qa2.x + qa2.y;
        statistics(stage, row + 1, more, qs, qa, [&] {
            // da, and the column sums of the post-norm and the gate
            const float e1 = qs * inv_n, e2 = qa * inv_n * ra * ra;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float2 o[P], qv[P], c[P];
                get_pairs(1, qw, s, qv);
                if constexpr (RELOAD) {
                    if (need_a) {
                        ln.load(m + at_a, p.a, row, s, c);
                        if (LAYER && post)
#pragma unroll
                            for (int j = 0; j < P; ++j) c[j] = __fadd2_rn(c[j], both(-mean_a));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < P; ++j) c[j] = av[s * P + j];
                }
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const int k = s * P + j;
                    float2 q = __fmul2_rn(d[k], qv[j]);
                    if (need_a) {
                        float2 ah = c[j];
                        if (post) {
                            q = __ffma2_rn(c[j], both(-e2), q);
                            if constexpr (LAYER) q = __fadd2_rn(q, both(-e1));
                            q = __fmul2_rn(q, both(ra));
                            ah = __fmul2_rn(c[j], both(ra));
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
        ++row;
    };
    // Which form the loop takes only decides how well it compiles: rows that follow one another in an inner loop that a far
    // row leaves (8192 x 4096 f32 129 us against 165, 6039 x 2560 f16 60 against 68), or one loop that tests each
    // row (16384 x 2048 bf16 94 us against 97, 8192 x 2049 bf16 181 against 195).
    if constexpr (LAYER && (SPARAM || sizeof(T) == 4)) {
        do {
            if (far_h || far_a) take_again();
            do one_row();
            while (row < slab.end && !(far_h || far_a));
        } while (row < slab.end);
    } else {
        while (row < slab.end) {
            if constexpr (LAYER) {
                if (__any_sync(kFull, far_h || far_a)) take_again();
            }
            one_row();
        }
    }
    if (p.sums) {
        float* part = p.part + index * V * cols + col0;
        auto slot_of = [&](const float2* v, int s, float2 (&o)[P]) {
#pragma unroll
            for (int j = 0; j < P; ++j) o[j] = v[s * P + j];
        };
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float2 o[P];
            slot_of(sum0, s, o);
            if (pre) ln.put_floats(part, s, o);
            slot_of(sumA, s, o);
            if (p.slices > 0) ln.put_floats(part + cols, s, o);
            if constexpr (LAYER) {
                slot_of(sum1, s, o);
                if (pre) ln.put_floats(part + 2 * cols, s, o);
                slot_of(sumB, s, o);
                if (p.slices > 0) ln.put_floats(part + 3 * cols, s, o);
            }
        }
    }
    ex.finish(p.debug);
}

// ---- host side -------------------------------------------------------------

template <class T, bool LAYER, int S, int LAYOUT, bool CLUSTER, int MODE, int THREADS, int CTAS, bool SPARAM = false>
cudaError_t bwd_go(const BlockBwArgs& in, const RowShape& shape, cudaStream_t stream) {
    BlockBwArgs a = in;
    RowShape g = shape;
    if (!SPARAM) g.params = 0;
    if (CLUSTER) {
        if (!(a.err = device_error_word())) return cudaErrorInvalidValue;
        a.debug = debug_flags_now();
        a.start = a.debug & kDebugExpirePeers ? NAN : 0.0f;
    }
    const int threads = g.teams * g.warps * 32;
    const size_t smem = row_smem(g);
    const auto kernel = bwd_kernel<T, LAYER, S, LAYOUT, CLUSTER, MODE, THREADS, CTAS, SPARAM>;
    const int64_t ctas = resident_ctas(reinterpret_cast<const void*>(kernel), threads, smem, g.cluster);
    if (ctas < 1) return cudaErrorInvalidConfiguration;
    block_slabs(&a, std::min(ctas * g.teams / g.cluster, block_slab_limit(a.rows, a.cols)));
    const unsigned grid = static_cast<unsigned>((a.slabs + g.teams - 1) / g.teams * g.cluster);
    cudaError_t e = launch_dependent(kernel, dim3(grid), threads, smem, g.cluster, stream, a, g);
    if (e != cudaSuccess || !a.sums) return e;
    return launch_block_finish(LAYER ? TR_NORM_LAYER : TR_NORM_RMS, a, stream);
}

// Full rows of one CTA are compiled for each pair of norms. 128 registers a thread let two CTAs of 256 threads
// share an SM; CTAs of 9 or 10 warps are compiled for two an SM with 96, against one an SM with 128: RMSNorm
// 6039 x 2560 f16 42 us against 46, 8192 x 2304 bf16 45 against 52, LayerNorm 6039 x 2560 f16 60 against 66,
// 6039 x 1280 f32 38 against 45; with few rows (RMSNorm 768 x 2560 bf16) it loses, 11.7 against 10.5.
// 16-bit ones take their parameters from shared memory: kept in those 96 registers, RMSNorm's two take 45 and 52 us.
template <class T, bool LAYER, int S, int MODE>
cudaError_t bwd_full(const BlockBwArgs& a, const RowShape& g, cudaStream_t stream) {
    if constexpr (S == 1) {
        if (g.teams * g.warps > 8 && g.teams * g.warps <= 10) return bwd_go<T, LAYER, S, LAYOUT_FULL, false, MODE, 320, 2, sizeof(T) == 2>(a, g, stream);
    }
    return bwd_go<T, LAYER, S, LAYOUT_FULL, false, MODE, 512, 1>(a, g, stream);
}

template <class T, bool LAYER, int S>
cudaError_t bwd_slots(int layout, const BlockBwArgs& a, const RowShape& g, cudaStream_t stream) {
    if (g.cluster > 1) {
        if constexpr (cluster_slots<T>(S, kBwdColumns)) {
            if (layout == LAYOUT_FULL) return bwd_go<T, LAYER, S, LAYOUT_FULL, true, 0, 512, 1>(a, g, stream);
            if (layout == LAYOUT_ALIGNED) return bwd_go<T, LAYER, S, LAYOUT_ALIGNED, true, 0, 512, 1>(a, g, stream);
            return bwd_go<T, LAYER, S, LAYOUT_ODD, true, 0, 512, 1>(a, g, stream);
        }
        return cudaErrorInvalidConfiguration;
    }
    if (layout == LAYOUT_ODD) return bwd_go<T, LAYER, S, LAYOUT_ODD, false, 0, 512, 1>(a, g, stream);
    if (layout == LAYOUT_ALIGNED) return bwd_go<T, LAYER, S, LAYOUT_ALIGNED, false, 0, 512, 1>(a, g, stream);
    if (a.pre && a.post) return bwd_full<T, LAYER, S, TR_BLOCK_PRE | TR_BLOCK_POST>(a, g, stream);
    return a.pre ? bwd_full<T, LAYER, S, TR_BLOCK_PRE>(a, g, stream) : bwd_full<T, LAYER, S, TR_BLOCK_POST>(a, g, stream);
}

template <class T, bool LAYER>
cudaError_t bwd_kind(const BlockBwArgs& a, bool* done, cudaStream_t stream) {
    const int tensors = (a.pre ? 2 : 0) + (a.post || a.dgate ? 1 : 0) + (a.dh ? 1 : 0);
    const bool odd = !rows_aligned(static_cast<int64_t>(a.cols) * static_cast<int>(sizeof(T)),
                                   {a.pre ? a.h : nullptr, a.pre ? a.dy : nullptr, a.post || a.dgate ? a.a : nullptr, a.dh, a.dx, a.da});
    int slots = 0;
    const RowShape g = row_shape<T>(a.cols, tensors, odd, LAYER, 4, sizeof(T) == 2 ? 64 : 0, kBwdColumns, &slots);
    *done = g.warps > 0;
    if (!*done) return cudaSuccess;
    const int layout = odd ? LAYOUT_ODD : row_full<T>(g, a.cols, slots) ? LAYOUT_FULL : LAYOUT_ALIGNED;
    if constexpr (sizeof(T) == 4) {
        if (slots == 2) return bwd_slots<T, LAYER, 2>(layout, a, g, stream);
    }
    return bwd_slots<T, LAYER, 1>(layout, a, g, stream);
}

}  // namespace block
}  // namespace tr
