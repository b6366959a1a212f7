// Norms over a list of tensors: host/device interface.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime.h>

#include "tr.h"

namespace tr {

constexpr int kListThreads = 256;
constexpr int kListTileBytes = 16 * 1024;  // four 16-byte loads a thread
constexpr int kListMax = 1000;             // tensors of one launch (kernel parameters hold 32764 bytes)
constexpr int kListFew = 64;               // launches of so few tensors carry a short parameter block
constexpr int kListMaxCtas = 1024;         // partials of one launch

// `count` tensors by value. Tensor i has the tiles first[i] .. first[i + 1] - 1 of the
// launch, each kListTileBytes of memory counted from its 16-byte boundary at or before `in`.
template <int N>
struct TensorList {
    const char* in[N];
    char* out[N];
    int64_t numel[N];
    uint32_t first[N + 1];
    uint8_t dtype[N];
    int count;
};

inline int64_t list_launches(int64_t count) { return count < 1 ? 1 : (count + kListMax - 1) / kListMax; }

// One partial norm a CTA (the sum of squares, or the largest magnitude).
// *ctas: the partials written, from `part` on; again: the list is scaled next (its end is kept in L2).
cudaError_t launch_list_norm(int kind, const TensorList<kListMax>& list, double* part, bool again, int* ctas,
                             cudaStream_t stream);
// The norm from n partials.
cudaError_t launch_list_total(int kind, const double* part, int n, float* norm, cudaStream_t stream);
// out = in * min(1, max_norm / (norm + eps)); with n partials the norm is theirs (and is
// written to *norm when `write`), otherwise *norm.
cudaError_t launch_list_scale(int kind, const TensorList<kListMax>& list, const double* part, int n, float* norm,
                              int write, float max_norm, float eps, cudaStream_t stream);

}  // namespace tr
