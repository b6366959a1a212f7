// Block norms: host/device interface of the gated residual norm and its backward.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime.h>

#include "tr.h"

namespace tr {

// h = rs x + bs gate post(a), y = pre(h); see tr.h. Absent vectors are null.
struct BlockArgs {
    const void* x;
    const void* a;  // the branch
    void* h;
    void* y;
    const float* post_w;
    const float* post_b;
    const float* gate;
    const float* pre_w;
    const float* pre_b;
    int64_t rows;
    int64_t group_rows;  // rows that share a gate row (rows when there is no gate)
    int cols;
    int post, pre;  // which norms there are
    float rs, bs, eps;
    unsigned* err;  // device error word (clusters' bounded waits; set by the launch)
    int debug;      // testing modes (kDebugModes) of those waits; set by the launch
    float start;    // what those exchanges' sums start from (0; see Exchange); set by the launch
};

struct BlockBwArgs {
    const void* h;
    const void* a;
    const void* dy;
    const void* dh;
    void* dx;
    void* da;
    const float* post_w;
    const float* post_b;
    const float* gate;
    const float* pre_w;
    float* dgate;
    float* dpost_w;
    float* dpost_b;
    float* dpre_w;
    float* dpre_b;
    int64_t rows;
    int64_t group_rows;
    int64_t groups;   // gate rows (1 when there is no gate)
    int64_t slices;   // slabs per group (0: each slab takes whole groups)
    int64_t slabs;    // row slabs, each with its own column partials
    int cols;
    int post, pre;
    int sums;         // column gradients are wanted
    float rs, bs, eps;
    float* stats;     // re-read path: kBlockStats floats a row
    float* part;      // slabs x vectors x cols partial column sums
    unsigned* err;    // device error word (clusters' bounded waits; set by the launch)
    int debug;        // testing modes (kDebugModes) of those waits; set by the launch
    float start;      // what those exchanges' sums start from (0; see Exchange); set by the launch
};

// The rows of a slab. With slices > 0 a slab is one of the `slices` equal parts
// of a group's rows, so its sums belong to one gate row; otherwise it is a run of
// whole groups, and the kernel finishes each group's gate gradient by itself.
struct SlabRows {
    int64_t begin, end;
};
__host__ __device__ inline SlabRows slab_rows(const BlockBwArgs& a, int64_t s) {
    if (a.slices > 0) {
        const int64_t g = s / a.slices, i = s % a.slices;
        return SlabRows{g * a.group_rows + a.group_rows * i / a.slices, g * a.group_rows + a.group_rows * (i + 1) / a.slices};
    }
    return SlabRows{a.groups * s / a.slabs * a.group_rows, a.groups * (s + 1) / a.slabs * a.group_rows};
}

constexpr int kBlockStats = 8;      // mean h, 1/sigma h, mean u, mean u hh, mean a, 1/sigma a (padded)
// Column-partial vectors of a slab: sum dy hh, sum D ah (or gate D ah), and for
// LayerNorm sum dy and sum D (or gate D) too.
inline int block_vectors(int kind) { return kind == TR_NORM_LAYER ? 4 : 2; }

// The most slabs a backward pass uses. A slab costs block_vectors() x cols floats: short
// rows may have many (teams of one warp, several a CTA), rows of up to 16384 columns two for each of
// 160 SMs, longer ones 2^22 floats a vector in all.
inline int64_t block_slab_limit(int64_t rows, int64_t cols) {
    int64_t n = cols > 16384 ? (1LL << 22) / cols : (1LL << 20) / cols;
    if (cols <= 16384) n = n < 320 ? 320 : (n > 4096 ? 4096 : n);
    if (n < 1) n = 1;
    return n < rows ? n : (rows < 1 ? 1 : rows);
}

// Choose the slabs for at most `target` of them.
inline void block_slabs(BlockBwArgs* a, int64_t target) {
    if (target < 1) target = 1;
    int64_t s = target / a->groups;
    if (s > a->group_rows) s = a->group_rows;
    if (s < 2 && a->groups > 1) {  // whole groups
        a->slices = 0;
        a->slabs = target < a->groups ? target : a->groups;
    } else {
        a->slices = s < 1 ? 1 : s;
        a->slabs = a->groups * a->slices;
    }
}

// CTAs (1 .. 8) of a row in the kernels that read rows again for each pass: as many as keep about 152 SMs
// busy with few rows, but no fewer than 4096 columns each.
inline int read_cluster(int64_t rows, int64_t cols) {
    int n = 1;
    while (n < 8 && rows * n * 2 <= 152 && cols / (n * 2) >= 4096) n *= 2;
    return n;
}

cudaError_t launch_block_forward(int kind, int dtype, const BlockArgs& a, cudaStream_t stream);
cudaError_t launch_block_backward(int kind, int dtype, const BlockBwArgs& a, cudaStream_t stream);
// The forward of rows that fit on the chip; *done is false (and nothing launched) for others.
cudaError_t launch_block_forward_f32(int kind, const BlockArgs& a, bool* done, cudaStream_t stream);
cudaError_t launch_block_forward_bf16(int kind, const BlockArgs& a, bool* done, cudaStream_t stream);
cudaError_t launch_block_forward_f16(int kind, const BlockArgs& a, bool* done, cudaStream_t stream);
// The backward of rows that fit on the chip; *done is false (and nothing launched) for others.
cudaError_t launch_block_backward_f32(int kind, const BlockBwArgs& a, bool* done, cudaStream_t stream);
cudaError_t launch_block_backward_bf16(int kind, const BlockBwArgs& a, bool* done, cudaStream_t stream);
cudaError_t launch_block_backward_f16(int kind, const BlockBwArgs& a, bool* done, cudaStream_t stream);
// The column gradients from the slabs' partials.
cudaError_t launch_block_finish(int kind, const BlockBwArgs& a, cudaStream_t stream);

}  // namespace tr
