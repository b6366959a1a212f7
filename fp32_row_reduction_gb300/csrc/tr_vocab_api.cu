// C-ABI of the embedding and of the linear cross entropy: argument checks on the host, then the
// launches. No entry point allocates device memory, waits, or lets a C++ exception out.
#include <cuda_runtime.h>

#include <cmath>

#include "tr.h"
#include "tr_check.h"
#include "tr_vocab.h"

namespace tr {
namespace {

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1024;  // tokens, rows and vocabularies are 32 bits in the kernels

bool is_dtype(int d) { return d == TR_F32 || d == TR_BF16 || d == TR_F16; }

tr_status check_order(const char* w, int order) {
    if (order < TR_ORDER_UNORDERED_TREE || order > TR_ORDER_FOLD_RIGHT)
        return fail(TR_ERR_INVALID_ARG, w, "order must be one of the tr_order values");
    if (order != TR_ORDER_UNORDERED_TREE) return fail(TR_ERR_UNSUPPORTED, w, "only the unordered policy is taken");
    return TR_OK;
}

tr_status check_embedding_sizes(const char* w, int64_t tokens, int64_t vocab, int64_t cols) {
    if (tokens < 0 || tokens > kMaxRows) return fail(TR_ERR_INVALID_ARG, w, "tokens must be in [0, 2^31 - 1024]");
    if (vocab < 1 || vocab > kMaxRows) return fail(TR_ERR_INVALID_ARG, w, "vocab must be in [1, 2^31 - 1024]");
    if (cols < 1 || cols >= (1 << 24)) return fail(TR_ERR_INVALID_ARG, w, "cols must be in [1, 2^24 - 1]");
    return TR_OK;
}

tr_status check_loss_sizes(const char* w, int64_t rows, int64_t cols, int64_t vocab) {
    if (rows < 0 || rows > kMaxRows) return fail(TR_ERR_INVALID_ARG, w, "rows must be in [0, 2^31 - 1024]");
    if (cols < 1 || cols >= (1 << 24)) return fail(TR_ERR_INVALID_ARG, w, "cols must be in [1, 2^24 - 1]");
    if (vocab < 1 || vocab >= (1 << 24)) return fail(TR_ERR_INVALID_ARG, w, "vocab must be in [1, 2^24 - 1]");
    return TR_OK;
}

tr_status check_loss(const char* w, int dtype, const void* weight, int64_t rows, int64_t cols, int64_t vocab, float scale, int order) {
    if (!is_dtype(dtype)) return fail(TR_ERR_INVALID_ARG, w, "dtype must be a tr_dtype");
    if (dtype == TR_F32)
        return fail(TR_ERR_UNSUPPORTED, w, "hidden and weight must be bfloat16 or float16: float32 products are not offered");
    tr_status s = check_order(w, order);
    if (s == TR_OK) s = check_loss_sizes(w, rows, cols, vocab);
    if (s != TR_OK) return s;
    if (!std::isfinite(scale)) return fail(TR_ERR_INVALID_ARG, w, "logit_scale must be finite");
    if (cols % 8 == 0 && reinterpret_cast<uintptr_t>(weight) % 16 != 0)
        return fail(TR_ERR_INVALID_ARG, w, "weight must be 16-byte aligned when cols is a multiple of 8");
    return TR_OK;
}

}  // namespace
}  // namespace tr

using namespace tr;

extern "C" {

tr_status tr_embedding(tr_dtype dtype, const void* table, const int64_t* ids, void* out, int64_t tokens, int64_t vocab,
                       int64_t cols, float scale, cudaStream_t stream) {
    static const char* w = "embedding";
    if (!is_dtype(dtype)) return fail(TR_ERR_INVALID_ARG, w, "dtype must be a tr_dtype");
    tr_status s = check_embedding_sizes(w, tokens, vocab, cols);
    if (s != TR_OK) return s;
    if (!std::isfinite(scale)) return fail(TR_ERR_INVALID_ARG, w, "scale must be finite");
    if (tokens == 0) return TR_OK;
    if (!table || !ids || !out) return fail(TR_ERR_INVALID_ARG, w, "table, ids and out must not be null");
    const size_t eb = element_bytes(dtype), row = eb * static_cast<size_t>(cols);
    const Range in[] = {{table, row * static_cast<size_t>(vocab), eb}, {ids, 8 * static_cast<size_t>(tokens), 8}};
    const Range to[] = {{out, row * static_cast<size_t>(tokens), eb}};
    s = check_ranges(w, in, to);
    if (s != TR_OK) return s;
    const EmbedArgs a{table, ids, out, tokens, vocab, static_cast<int>(cols), scale};
    return guarded(w, [&] { return cuda_status(launch_embedding(dtype, a, stream), w); });
}

tr_status tr_embedding_backward_workspace_bytes(int64_t tokens, int64_t cols, size_t* bytes) {
    static const char* w = "embedding backward workspace";
    if (!bytes) return fail(TR_ERR_INVALID_ARG, w, "bytes must not be null");
    const tr_status s = check_embedding_sizes(w, tokens, 1, cols);
    if (s != TR_OK) return s;
    *bytes = EmbedGradPlan(tokens, cols).bytes;
    return TR_OK;
}

tr_status tr_embedding_backward(tr_dtype dtype, tr_dtype grad_dtype, const void* dy, const int64_t* ids, void* dtable,
                                int64_t tokens, int64_t vocab, int64_t cols, float scale, int32_t accumulate, tr_order order,
                                void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    static const char* w = "embedding backward";
    if (!is_dtype(dtype)) return fail(TR_ERR_INVALID_ARG, w, "dtype must be a tr_dtype");
    if (grad_dtype != dtype && grad_dtype != TR_F32)
        return fail(TR_ERR_INVALID_ARG, w, "grad_dtype must be dtype or TR_F32");
    tr_status s = check_order(w, order);
    if (s == TR_OK) s = check_embedding_sizes(w, tokens, vocab, cols);
    if (s != TR_OK) return s;
    if (!std::isfinite(scale)) return fail(TR_ERR_INVALID_ARG, w, "scale must be finite");
    if (accumulate != 0 && accumulate != 1) return fail(TR_ERR_INVALID_ARG, w, "accumulate must be 0 or 1");
    if (!dtable) return fail(TR_ERR_INVALID_ARG, w, "dtable must not be null");
    const size_t eb = element_bytes(dtype), gb = element_bytes(grad_dtype), n = static_cast<size_t>(cols);
    const Range in[] = {{dy, eb * n * static_cast<size_t>(tokens), eb}, {ids, 8 * static_cast<size_t>(tokens), 8}};
    const Range out[] = {{dtable, gb * n * static_cast<size_t>(vocab), gb}, {workspace, tokens > 0 ? workspace_bytes : 0, 16}};
    s = check_ranges(w, in, out);
    if (s != TR_OK) return s;
    if (tokens == 0) {  // empty sums
        if (accumulate) return TR_OK;
        return cuda_status(cudaMemsetAsync(dtable, 0, out[0].bytes, stream), w);
    }
    if (!dy || !ids) return fail(TR_ERR_INVALID_ARG, w, "dy and ids must not be null");
    if (!workspace || workspace_bytes < EmbedGradPlan(tokens, cols).bytes)
        return fail(TR_ERR_INVALID_ARG, w, "the workspace is missing or smaller than tr_embedding_backward_workspace_bytes");
    const EmbedGradArgs a{dy, ids, dtable, tokens, vocab, static_cast<int>(cols), scale, accumulate, static_cast<char*>(workspace)};
    return guarded(w, [&] { return cuda_status(launch_embedding_backward(dtype, grad_dtype, a, stream), w); });
}

tr_status tr_linear_cross_entropy_workspace_bytes(int64_t rows, int64_t cols, int64_t vocab, int32_t backward, size_t* bytes) {
    static const char* w = "linear cross entropy workspace";
    if (!bytes) return fail(TR_ERR_INVALID_ARG, w, "bytes must not be null");
    if (backward != 0 && backward != 1) return fail(TR_ERR_INVALID_ARG, w, "backward must be 0 or 1");
    const tr_status s = check_loss_sizes(w, rows, cols, vocab);
    if (s != TR_OK) return s;
    *bytes = rows > 0 ? LossPlan(rows, cols, vocab, backward != 0).bytes : 0;
    return TR_OK;
}

tr_status tr_linear_cross_entropy(tr_dtype dtype, const void* hidden, const void* weight, const int64_t* labels, float* losses,
                                  float* lse, int64_t rows, int64_t cols, int64_t vocab, float logit_scale, int64_t ignore_label,
                                  tr_order order, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    static const char* w = "linear cross entropy";
    tr_status s = check_loss(w, dtype, weight, rows, cols, vocab, logit_scale, order);
    if (s != TR_OK) return s;
    if (rows == 0) return TR_OK;
    if (!hidden || !weight || !labels || !losses)
        return fail(TR_ERR_INVALID_ARG, w, "hidden, weight, labels and losses must not be null");
    const size_t n = static_cast<size_t>(cols) * 2, r = static_cast<size_t>(rows);
    const Range in[] = {{hidden, n * r, 2}, {weight, n * static_cast<size_t>(vocab), 2}, {labels, 8 * r, 8}};
    const Range out[] = {{losses, 4 * r, 4}, {lse, 4 * r, 4}, {workspace, workspace_bytes, 16}};
    s = check_ranges(w, in, out);
    if (s != TR_OK) return s;
    if (!workspace || workspace_bytes < LossPlan(rows, cols, vocab, false).bytes)
        return fail(TR_ERR_INVALID_ARG, w, "the workspace is missing or smaller than tr_linear_cross_entropy_workspace_bytes");
    LossArgs a{};
    a.hidden = hidden;
    a.weight = weight;
    a.labels = labels;
    a.losses = losses;
    a.lse = lse;
    a.rows = rows;
    a.vocab = vocab;
    a.ignore = ignore_label;
    a.cols = static_cast<int>(cols);
    a.logit_scale = logit_scale;
    a.ws = static_cast<char*>(workspace);
    return guarded(w, [&] { return cuda_status(launch_loss(dtype, a, stream), w); });
}

tr_status tr_linear_cross_entropy_backward(tr_dtype dtype, const void* hidden, const void* weight, const int64_t* labels,
                                           const float* lse, const float* dloss, const float* dlse, void* dhidden, void* dweight,
                                           int64_t rows, int64_t cols, int64_t vocab, float logit_scale, int64_t ignore_label,
                                           tr_order order, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    static const char* w = "linear cross entropy backward";
    tr_status s = check_loss(w, dtype, weight, rows, cols, vocab, logit_scale, order);
    if (s != TR_OK) return s;
    if (!dhidden && !dweight) return fail(TR_ERR_INVALID_ARG, w, "dhidden and dweight must not both be null");
    const size_t n = static_cast<size_t>(cols) * 2, r = static_cast<size_t>(rows), table = n * static_cast<size_t>(vocab);
    const Range in[] = {{hidden, n * r, 2}, {weight, rows ? table : 0, 2}, {labels, 8 * r, 8}, {lse, 4 * r, 4}, {dloss, 4 * r, 4},
                        {dlse, 4 * r, 4}};
    const Range out[] = {{dhidden, n * r, 2}, {dweight, table, 2}, {workspace, rows ? workspace_bytes : 0, 16}};
    s = check_ranges(w, in, out);
    if (s != TR_OK) return s;
    if (rows == 0) return dweight ? cuda_status(cudaMemsetAsync(dweight, 0, table, stream), w) : TR_OK;  // empty sums
    if (!hidden || !weight || !labels || !lse)
        return fail(TR_ERR_INVALID_ARG, w, "hidden, weight, labels and lse must not be null");
    if (!workspace || workspace_bytes < LossPlan(rows, cols, vocab, true).bytes)
        return fail(TR_ERR_INVALID_ARG, w, "the workspace is missing or smaller than tr_linear_cross_entropy_workspace_bytes");
    LossArgs a{};
    a.hidden = hidden;
    a.weight = weight;
    a.labels = labels;
    a.lse_in = lse;
    a.dloss = dloss;
    a.dlse = dlse;
    a.dhidden = dhidden;
    a.dweight = dweight;
    a.rows = rows;
    a.vocab = vocab;
    a.ignore = ignore_label;
    a.cols = static_cast<int>(cols);
    a.logit_scale = logit_scale;
    a.ws = static_cast<char*>(workspace);
    return guarded(w, [&] { return cuda_status(launch_loss_backward(dtype, a, stream), w); });
}

}  // extern "C"
