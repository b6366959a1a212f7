// The vocabulary's two ends (embedding, linear cross entropy): host/device interface.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime.h>

#include "tr.h"

namespace tr {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// ---- embedding ------------------------------------------------------------------

struct EmbedArgs {
    const void* table;
    const int64_t* ids;
    void* out;
    int64_t tokens, vocab;
    int cols;
    float scale;
};
cudaError_t launch_embedding(int dtype, const EmbedArgs& a, cudaStream_t stream);

constexpr int kSortTile = 16384;  // keys that one CTA sorts
constexpr int kPassTile = 4096;   // keys of a CTA where several sort
constexpr int kSortBins = 256;
constexpr int kSumTile = 32;      // sorted tokens of a warp of the sums

// Workspace of the gradient, in this order: the sorted ids and the tokens they belong to (each twice, the
// passes of a sort over several CTAs go to and fro), the sort's counts, the list of the long
// segments, and their partial sums.
struct EmbedGradPlan {
    int64_t sort_tiles, sum_tiles;
    size_t keys[2], places[2], counts, listed, partials, bytes;  // offsets
    EmbedGradPlan(int64_t tokens, int64_t cols) {
        sort_tiles = tokens <= kSortTile ? 1 : ceil_div(tokens, kPassTile);
        sum_tiles = ceil_div(tokens, kSumTile);
        const int copies = sort_tiles > 1 ? 2 : 1;
        size_t at = 0;
        auto take = [&](size_t n) {
            const size_t here = at;
            at += (n + 255) / 256 * 256;
            return here;
        };
        for (int i = 0; i < 2; ++i) keys[i] = i < copies ? take(4 * static_cast<size_t>(tokens)) : keys[0];
        for (int i = 0; i < 2; ++i) places[i] = i < copies ? take(4 * static_cast<size_t>(tokens)) : places[0];
        counts = sort_tiles > 1 ? take(4 * static_cast<size_t>(sort_tiles) * kSortBins) : at;
        listed = take(4 * static_cast<size_t>(sum_tiles + 1));
        partials = take(8 * static_cast<size_t>(sum_tiles) * round_up(cols, 8));
        bytes = tokens > 0 ? at : 0;
    }
};

struct EmbedGradArgs {
    const void* dy;
    const int64_t* ids;
    void* dtable;
    int64_t tokens, vocab;
    int cols;
    float scale;
    int accumulate;
    char* ws;
};
cudaError_t launch_embedding_backward(int dtype, int grad_dtype, const EmbedGradArgs& a, cudaStream_t stream);

// ---- linear cross entropy ---------------------------------------------------------

constexpr int kTileRows = 256;  // packed rows come in whole tiles

// Packed rows: the rows that have a loss, in order. Workspace of both directions:
struct LossPlan {
    int64_t rows_pad;  // packed rows at most, in whole tiles
    int64_t pitch;     // elements of a packed row of hidden (or of weight)
    int64_t piece;     // backward: columns of the vocabulary at a time
    int64_t parts;     // forward: partial (maximum, sum) pairs of a row
    int width;         // words of a tile of logits
    int grad_width;    // columns of a tile of the gradients
    int splits;        // of the depth of the hidden gradient
    int logit_part;    // blocks of the width that the logits are summed over at once, the same in both directions
    bool parted;       // whether a depth of the gradients is summed in parts
    bool fine_hidden, fine_weight;  // whether a gradient's products take dz in two terms
    int terms;         // of dz that are kept
    size_t head, map, labels, lse, coef, onehot, hidden, weight, parts_at, picked, probs, sums, bytes;
    bool pack_weight;  // rows of the weight that do not start on 16 bytes are copied to ones that do
    LossPlan(int64_t rows, int64_t cols, int64_t vocab, bool backward);
};

// What the first CTA finds out about the rows.
struct LossHead {
    int64_t count;  // rows that have a loss
    float scale;    // backward: 2^14 / the largest |dloss|, or 2^15 / the largest |dloss| + |dlse| where that is over twice as large
    float unscale;  // logit_scale / scale
};

struct LossArgs {
    const void* hidden;
    const void* weight;
    const int64_t* labels;
    float* losses;  // forward
    float* lse;     // forward: written (or null)
    const float* lse_in;
    const float* dloss;
    const float* dlse;
    void* dhidden;
    void* dweight;
    int64_t rows, vocab, ignore;
    int cols;
    float logit_scale;
    char* ws;
};
cudaError_t launch_loss(int dtype, const LossArgs& a, cudaStream_t stream);
cudaError_t launch_loss_backward(int dtype, const LossArgs& a, cudaStream_t stream);

}  // namespace tr
