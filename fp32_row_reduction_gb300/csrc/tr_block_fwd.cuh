// The gated residual norm with the rows on chip: h = rs x + bs gate post(a), y = pre(h).
//
// HBM-bound: x and a are read, h and y written once (16384 x 4096 bf16: RMSNorm 83 us, 95% of the measured copy rate,
// LayerNorm 89 us). A row's y waits for the statistics of h, which
// wait for those of a; so that a row costs one exchange between its warps, the sum over h of a row
// travels with the sum over a of the next one. LayerNorm's sums are taken about a shift that each warp
// finds for itself (lane_mean; for h from the same elements' own x and a), and once more for a row whose shift is far
// from its mean. The parameters of a thread's columns
// stay in its registers for all its rows.
#pragma once

#include "tr_block_rows.cuh"

namespace tr {
namespace block {

template <class T, bool LAYER, int S, int LAYOUT, bool CLUSTER, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) fwd_kernel(const BlockArgs p, const RowShape g, const int64_t slabs) {
    constexpr int E = 16 / static_cast<int>(sizeof(T));
    constexpr int P = E / 2;  // pairs of a slot
    constexpr int K = S * P;  // pairs of a thread
    constexpr bool ODD = LAYOUT == LAYOUT_ODD;
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
    Exchange<CLUSTER, LAYER ? 4 : 2> ex(team_smem, g.warps * g.cluster, rank * g.warps + (t >> 5), team, g.warps, p.err, p.start);
    ex.init();
    const int stage_bytes = g.tensors * g.tensor_bytes;
    const RowStart<T, LAYOUT, CLUSTER> row_start(cols, ln.row_bytes);  // LayerNorm's
    char* starts = team_smem + exchange_bytes(g) + (t >> 5) * g.stages * g.sampled;
    char* ring = reinterpret_cast<char*>(smem) + fixed_bytes(g) + team * g.stages * stage_bytes;
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
            if constexpr (LAYER) {
                row_start.fetch(p.a, row, starts + stage * g.sampled);
                if (p.pre) row_start.fetch(p.x, row, starts + stage * g.sampled + kRowStartBytes);
            }
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
    float2 gb[LAYER ? K : 1], b[LAYER ? K : 1];  // bs gate b_post;  the pre-norm's bias
#pragma unroll
    for (int s = 0; s < S; ++s) {
        float2 v[P];
        ln.param(at0(p.pre_w), s, 1.0f, v);
#pragma unroll
        for (int j = 0; j < P; ++j) w[s * P + j] = v[j];
        if constexpr (LAYER) {
            ln.param(at0(p.pre_b), s, 0.0f, v);
#pragma unroll
            for (int j = 0; j < P; ++j) b[s * P + j] = v[j];
        }
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
            if constexpr (LAYER) {
                ln.param(at0(p.post_b), s, 0.0f, o);
#pragma unroll
                for (int j = 0; j < P; ++j) gb[s * P + j] = __fmul2_rn(v[j], __fmul2_rn(both(p.bs), o[j]));
            }
        }
    };
    // LayerNorm: the parameters at the lane's element of a row's start: bs gate w_post, bs gate b_post
    const int probe = static_cast<int>(threadIdx.x & 31) % cols;
    float probe_w = 1.0f, probe_b = 0.0f;
    auto enter_probe = [&](int64_t row) {
        const float gt = p.bs * (p.gate ? __ldg(p.gate + row / p.group_rows * cols + probe) : 1.0f);
        probe_w = gt * (p.post_w ? __ldg(p.post_w + probe) : 1.0f);
        probe_b = gt * (p.post_b ? __ldg(p.post_b + probe) : 0.0f);
    };

    float2 h[K];
    float ra = 1.0f, ma = 0.0f;  // of the row at work
    float rh = 1.0f, mh = 0.0f;
    bool far_h = false, far_a = false;  // LayerNorm: the row before's sums over h, and this row's over a, are to be taken again
    // the sums over h about sh (where `this_row`) and over a of row `row` staged at m about sa (where `next_row`):
    // squares of h and a, and for LayerNorm h and a
    auto sums_about = [&](const char* m, int64_t row, bool this_row, bool next_row, float sh, float sa, float (&sum)[LAYER ? 4 : 2]) {
        float2 hh = both(0.0f), aa = both(0.0f), h1 = both(0.0f), a1 = both(0.0f);
        auto shifted = [&](float2 v, float shift, bool xi, bool yi) {
            if constexpr (!LAYER) return v;
            float2 c = __fadd2_rn(v, both(-shift));
            if (!xi) c.x = 0.0f;
            if (!yi) c.y = 0.0f;
            return c;
        };
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (p.pre && this_row)
                ln.pairs(s, [&](int j, bool xi, bool yi) {
                    const float2 c = shifted(h[s * P + j], sh, xi, yi);
                    hh = __ffma2_rn(c, c, hh);
                    if constexpr (LAYER) h1 = __fadd2_rn(h1, c);
                });
            if (p.post && next_row) {
                float2 x[P];
                ln.load(m, p.a, row, s, x);
                ln.pairs(s, [&](int j, bool xi, bool yi) {
                    const float2 c = shifted(x[j], sa, xi, yi);
                    aa = __ffma2_rn(c, c, aa);
                    if constexpr (LAYER) a1 = __fadd2_rn(a1, c);
                });
            }
        }
        sum[0] = hh.x + hh.y;
        sum[1] = aa.x + aa.y;
        if constexpr (LAYER) {
            sum[2] = h1.x + h1.y;
            sum[3] = a1.x + a1.y;
        }
        ex.sums(sum);
    };
    auto statistics = [&](const char* m, int64_t row, bool this_row, bool next_row, float sh, float sa) {
        float v[LAYER ? 4 : 2];
        sums_about(m, row, this_row, next_row, sh, sa, v);
        float sq_h = v[0], sq_a = v[1];
        if constexpr (LAYER) {
            const float dh = v[2] * inv_n, da = v[3] * inv_n;  // the means, from the shifts
            sq_h = squares_about_mean(v[0], v[2], dh, far_h);
            sq_a = squares_about_mean(v[1], v[3], da, far_a);
            mh = sh + dh;
            if (p.post) ma = sa + da;
        }
        // rsqrtf is good to 2^-22, as the sums are
        rh = rsqrtf(fmaf(sq_h, inv_n, p.eps));
        if (p.post) ra = rsqrtf(fmaf(sq_a, inv_n, p.eps));
    };

    int64_t left = 0;  // rows of the running gate row still to come
    if (begin < end) {
        enter_group(begin);
        if constexpr (LAYER) enter_probe(begin);
        left = p.group_rows - begin % p.group_rows;
    }
    ring_wait(g.stages, 2);
    if constexpr (ODD) odd_barrier();
    float a_here = 0.0f;  // LayerNorm: the lane's element of a
    if constexpr (LAYER) {
        __syncwarp();
        a_here = row_start.get(p.a, begin, starts, ring);
    }
    if (p.post) statistics(ring, begin, false, true, 0.0f, LAYER ? lane_mean(a_here) : 0.0f);
    auto write_y = [&](int64_t row) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float2 o[P];
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int k = s * P + j;
                const float2 c = LAYER ? __fadd2_rn(h[k], both(-mh)) : h[k];
                const float2 n = __fmul2_rn(c, both(rh));
                o[j] = LAYER ? __ffma2_rn(n, w[k], b[LAYER ? k : 0]) : __fmul2_rn(n, w[k]);
            }
            ln.store(p.y, row, s, o);
        }
    };
    int stage = 0, fill = g.stages - 1;
    int64_t row = begin;
    // Sums about a shift too far from the mean are taken again about that mean (by all warps of the row alike) between two
    // rows, and the row before is normalised again. A test in the middle of a row's chain costs 16384 x 4096 bf16 12 us.
    auto take_again = [&]() {
        const bool again_h = far_h, again_a = far_a;
        const float here_ra = ra, here_ma = ma;
        statistics(ring + stage * stage_bytes, row, again_h, again_a, mh, ma);
        if (!again_a) {
            ra = here_ra;
            ma = here_ma;
        }
        if (again_h) write_y(row - 1);
        far_h = far_a = false;
    };
    auto one_row = [&]() {
        if (left == 0) {
            enter_group(row);
            if constexpr (LAYER) enter_probe(row);
            left = p.group_rows;
        }
        --left;
        if constexpr (ODD) {  // the next row is here, and every thread is done with the row before
            ring_wait(g.stages, 1);
            odd_barrier();
        }
        fetch(row + g.stages - 1, fill);
        fill = fill + 1 == g.stages ? 0 : fill + 1;
        [[maybe_unused]] const int here = stage;
        const char* m = ring + stage * stage_bytes;
        stage = stage + 1 == g.stages ? 0 : stage + 1;
        const char* next = ring + stage * stage_bytes;
        const bool more = row + 1 < end;
        float h_here = 0.0f;
        if constexpr (LAYER) {
            if (p.pre) {
                const float x_here = row_start.get(p.x, row, starts + here * g.sampled + kRowStartBytes, m + g.tensor_bytes);
                h_here = fmaf((a_here - ma) * ra, probe_w, fmaf(p.rs, x_here, probe_b));
            }
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float2 x[P], v[P];
            ln.load(m, p.a, row, s, v);
            ln.load(m + g.tensor_bytes, p.x, row, s, x);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int k = s * P + j;
                const float2 c = LAYER ? __fadd2_rn(v[j], both(-ma)) : v[j];
                const float2 n = __fmul2_rn(c, both(ra));
                h[k] = __ffma2_rn(n, gw[k], LAYER ? __ffma2_rn(both(p.rs), x[j], gb[LAYER ? k : 0]) : __fmul2_rn(both(p.rs), x[j]));
                if (!ln.in(s, 2 * j)) h[k].x = 0.0f;
                if (!ln.in(s, 2 * j + 1)) h[k].y = 0.0f;
                v[j] = h[k];
            }
            if (p.h) ln.store(p.h, row, s, v);
        }
        if constexpr (!ODD) ring_wait(g.stages, 2);
        float a_next = 0.0f;
        if constexpr (LAYER) {
            __syncwarp();
            if (more) a_next = row_start.get(p.a, row + 1, starts + stage * g.sampled, next);
        }
        statistics(next, row + 1, true, more, LAYER ? lane_mean(h_here) : 0.0f, LAYER ? lane_mean(a_next) : 0.0f);
        a_here = a_next;
        if (p.pre) write_y(row);
        ++row;
    };
    // Which form the loop takes only decides how well it compiles: rows that follow one another in an inner loop that a far
    // row leaves (2048 x 20000 bf16 103 us against 112, 8192 x 7000 f32 164 against 197), or one loop that
    // tests each row (16384 x 4096 bf16 89 us against 93, 8192 x 2049 bf16 73 against 78).
    if constexpr (LAYER && LAYOUT == LAYOUT_ALIGNED) {
        do {
            if (far_h || far_a) take_again();
            if (row < end) {
                do one_row();
                while (row < end && !(far_h || far_a));
            }
        } while (row < end || far_h || far_a);
    } else {
        for (;;) {
            if constexpr (LAYER) {
                if (__any_sync(kFull, far_h || far_a)) take_again();
            }
            if (row >= end) break;
            one_row();
        }
    }
    ex.finish(p.debug);
}

// ---- host side -------------------------------------------------------------

template <class T, bool LAYER, int S, int LAYOUT, bool CLUSTER, int THREADS, int CTAS>
cudaError_t fwd_go_with(const BlockArgs& in, const RowShape& g, cudaStream_t stream) {
    BlockArgs a = in;
    if (CLUSTER) {
        if (!(a.err = device_error_word())) return cudaErrorInvalidValue;
        a.debug = debug_flags_now();
        a.start = a.debug & kDebugExpirePeers ? NAN : 0.0f;
    }
    const int threads = g.teams * g.warps * 32;
    const size_t smem = row_smem(g);
    const auto kernel = fwd_kernel<T, LAYER, S, LAYOUT, CLUSTER, THREADS, CTAS>;
    const int64_t ctas = resident_ctas(reinterpret_cast<const void*>(kernel), threads, smem, g.cluster);
    if (ctas < 1) return cudaErrorInvalidConfiguration;
    const int64_t slabs = std::min(a.rows, ctas * g.teams / g.cluster);
    const unsigned grid = static_cast<unsigned>((slabs + g.teams - 1) / g.teams * g.cluster);
    return launch_dependent(kernel, dim3(grid), threads, smem, g.cluster, stream, a, g, slabs);
}

// 64 registers are enough for RMSNorm's rows (1024 threads an SM); LayerNorm's biases take more, so CTAs of at
// most 320 threads are compiled for two an SM, and larger ones run one.
template <class T, bool LAYER, int S, int LAYOUT, bool CLUSTER>
cudaError_t fwd_go(const BlockArgs& a, const RowShape& g, cudaStream_t stream) {
    if constexpr (!LAYER && S * 16 / sizeof(T) <= 8) {
        return fwd_go_with<T, LAYER, S, LAYOUT, CLUSTER, 512, 2>(a, g, stream);
    } else {
        if constexpr (!CLUSTER && S == 1) {
            // (16-bit rows of one slot have fewer than 1024 columns: 8 warps at most)
            if (sizeof(T) == 2 || g.teams * g.warps <= 10) return fwd_go_with<T, LAYER, S, LAYOUT, CLUSTER, 320, 2>(a, g, stream);
        }
        if constexpr (CLUSTER || S > 1 || sizeof(T) == 4) return fwd_go_with<T, LAYER, S, LAYOUT, CLUSTER, 512, 1>(a, g, stream);
        return cudaErrorInvalidConfiguration;
    }
}

template <class T, bool LAYER, int S, bool CLUSTER>
cudaError_t fwd_layout(int layout, const BlockArgs& a, const RowShape& g, cudaStream_t stream) {
    if (layout == LAYOUT_FULL) return fwd_go<T, LAYER, S, LAYOUT_FULL, CLUSTER>(a, g, stream);
    if (layout == LAYOUT_ALIGNED) return fwd_go<T, LAYER, S, LAYOUT_ALIGNED, CLUSTER>(a, g, stream);
    return fwd_go<T, LAYER, S, LAYOUT_ODD, CLUSTER>(a, g, stream);
}

template <class T, bool LAYER, int S>
cudaError_t fwd_slots(int layout, const BlockArgs& a, const RowShape& g, cudaStream_t stream) {
    if (g.cluster == 1) return fwd_layout<T, LAYER, S, false>(layout, a, g, stream);
    if constexpr (cluster_slots<T>(S, kFwdColumns)) return fwd_layout<T, LAYER, S, true>(layout, a, g, stream);
    return cudaErrorInvalidConfiguration;
}

template <class T, bool LAYER>
cudaError_t fwd_kind(const BlockArgs& a, bool* done, cudaStream_t stream) {
    const bool odd = !rows_aligned(static_cast<int64_t>(a.cols) * static_cast<int>(sizeof(T)), {a.x, a.a, a.h, a.y});
    int slots = 0;
    // a third stage is all RMSNorm wants (16384 x 4096 bf16: 84 us, with a fourth 94: more loads under way only
    // keep the stores waiting); LayerNorm's longer rows of work hide a little better behind four (89 us, with three 90)
    const RowShape g = row_shape<T>(a.cols, 2, odd, LAYER, LAYER ? 4 : 3, 0, kFwdColumns, &slots);
    *done = g.warps > 0;
    if (!*done) return cudaSuccess;
    const int layout = odd ? LAYOUT_ODD : row_full<T>(g, a.cols, slots) ? LAYOUT_FULL : LAYOUT_ALIGNED;
    if (slots == 2) return fwd_slots<T, LAYER, 2>(layout, a, g, stream);
    if constexpr (sizeof(T) == 4) {
        if (slots == 3) return fwd_slots<T, LAYER, 3>(layout, a, g, stream);
        if (slots == 4) return fwd_slots<T, LAYER, 4>(layout, a, g, stream);
    }
    return fwd_slots<T, LAYER, 1>(layout, a, g, stream);
}

}  // namespace block
}  // namespace tr
