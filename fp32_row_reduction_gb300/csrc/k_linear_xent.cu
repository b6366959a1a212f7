// Softmax cross entropy of logits = logit_scale hidden weight^T that are never kept, and its gradients.
//
// With z = log2(e) logits, forward: every row's maximum m and sum of 2^(z - m) over each tile of the vocabulary, which a
// last kernel joins: lse = ln 2 (m + log2 sum), loss = ln 2 (m - z_label) + ln sum.
// Backward, for one piece of the vocabulary after another: dz = (dloss + dlse) 2^(z - lse) - dloss [label], rounded to the
// inputs' type for the products dhidden += dz weight (in float32 over the pieces) and dweight = dz^T hidden.
#include <algorithm>
#include <cmath>

#include "tr_block.cuh"
#include "tr_launch.h"
#include "tr_vocab.h"

namespace tr {

LossPlan::LossPlan(int64_t rows, int64_t cols, int64_t vocab, bool backward) {
    size_t at = 0;
    auto take = [&](int64_t n) {
        const size_t here = at;
        at += (static_cast<size_t>(n) + 255) / 256 * 256;
        return here;
    };
    rows_pad = round_up(rows, kTileRows);
    pitch = round_up(cols, 8);
    parts = ceil_div(vocab, 64);
    pack_weight = cols % 8 != 0;
    // dz of a piece: 2^27 values (256 MB), and at least 4096 columns, so that the sums over the pieces cost little
    const int64_t most = std::max<int64_t>(4096, (int64_t{1} << 27) / rows_pad / 256 * 256);
    const int64_t pieces = ceil_div(vocab, std::min(most, round_up(vocab, 256)));
    piece = round_up(ceil_div(vocab, pieces), 256);
    head = take(sizeof(LossHead));
    map = take(rows_pad * 4);
    labels = take(rows_pad * 4);
    hidden = take(rows_pad * pitch * 2);
    weight = pack_weight ? take(vocab * pitch * 2) : at;
    lse = coef = onehot = probs = sums = parts_at = picked = at;
    if (backward) {
        lse = take(rows_pad * 4);
        coef = take(rows_pad * 4);
        onehot = take(rows_pad * 4);
        probs = take(rows_pad * piece * 2);
        sums = take(rows_pad * pitch * 4);
    } else {
        parts_at = take(parts * rows_pad * 8);
        picked = take(rows_pad * 4);
    }
    bytes = rows > 0 ? at : 0;
}

namespace loss {

using block::from_float;
using block::to_float;

constexpr int kThreads = 256;
constexpr int kScanThreads = 1024;

struct Ws {
    LossHead* head;
    int* map;
    int* labels;
    float* lse;
    float* coef;
    float* onehot;
    float2* parts;
    float* picked;
    float* sums;
    int64_t rows_pad;
};

// ---- the rows that have a loss -------------------------------------------------------

// One CTA lists them in order, with their labels (-1: outside the vocabulary) and, backward, their coefficients:
// of the probability (dloss + dlse) and of the label (dloss). The outputs of rows without a loss are zeros.
__global__ void __launch_bounds__(kScanThreads) rows_kernel(LossArgs a, Ws w, int backward) {
    __shared__ int warp_count[32];
    __shared__ float warp_most[32];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t count = 0;
    float most = 0.0f;
    for (int64_t r0 = 0; r0 < a.rows; r0 += kScanThreads) {
        const int64_t r = r0 + threadIdx.x;
        const int64_t label = r < a.rows ? a.labels[r] : a.ignore;
        const bool counted = r < a.rows && label != a.ignore;
        const unsigned votes = __ballot_sync(kFull, counted);
        __syncthreads();
        if (lane == 0) warp_count[warp] = __popc(votes);
        __syncthreads();
        const int mine = warp_count[lane];
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += v;
        }
        const int64_t at = count + __shfl_sync(kFull, inc - mine, warp) + __popc(votes & ((1u << lane) - 1u));
        count += __shfl_sync(kFull, inc, 31);
        if (counted) {
            w.map[at] = static_cast<int>(r);
            w.labels[at] = label >= 0 && label < a.vocab ? static_cast<int>(label) : -1;
            if (backward) {
                const float d = a.dloss ? a.dloss[r] : 1.0f, e = a.dlse ? a.dlse[r] : 0.0f;
                w.lse[at] = a.lse_in[r] * kL2E;
                w.coef[at] = d + e;
                w.onehot[at] = d;
                most = fmaxf(most, fabsf(d) + fabsf(e));
            }
        } else if (!backward && r < a.rows) {
            a.losses[r] = 0.0f;
            if (a.lse) a.lse[r] = 0.0f;
        }
    }
    most = warp_allreduce<MaxOp, 32>(most);
    if (lane == 0) warp_most[warp] = most;
    __syncthreads();
    if (warp == 0) {
        most = warp_allreduce<MaxOp, 32>(warp_most[lane]);
        if (lane == 0) {
            w.head->count = count;
            // dz times this is at most 2^15 and mostly above float16's smallest normal number
            int e = 0;
            if (most > 0.0f && most < INFINITY) frexpf(most, &e);
            e = max(-100, min(100, e));
            w.head->scale = ldexpf(1.0f, 15 - e);
            w.head->unscale = ldexpf(a.logit_scale, e - 15);
        }
    }
}

// Rows copied to rows of `pitch` elements that start on 16 bytes; map: which row each is (null: all, in order). Packed
// rows up to the next whole tile are zeros. Backward, the gradients of rows without a loss are zeros.
template <class T>
__global__ void __launch_bounds__(kThreads) pack_kernel(LossArgs a, Ws w, const T* src, int64_t rows, T* dst, int64_t pitch,
                                                        int64_t packed, T* zeros) {
    pdl_enter();
    const int64_t count = w.head && w.map ? w.head->count : rows;
    const int lane = threadIdx.x & 31, warps = kThreads / 32;
    const int64_t step = static_cast<int64_t>(gridDim.x) * warps;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * warps + (threadIdx.x >> 5); i < packed; i += step) {
        if (i >= (count + kTileRows - 1) / kTileRows * kTileRows) break;
        const T* row = i < count ? src + static_cast<int64_t>(w.map ? w.map[i] : i) * a.cols : nullptr;
        for (int c = lane; c < pitch; c += 32) dst[i * pitch + c] = row && c < a.cols ? row[c] : from_float<T>(0.0f);
    }
    if (!zeros) return;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * warps + (threadIdx.x >> 5); r < a.rows; r += step) {
        if (a.labels[r] != a.ignore) continue;
        for (int c = lane; c < a.cols; c += 32) zeros[r * a.cols + c] = from_float<T>(0.0f);
    }
}

// ---- products -------------------------------------------------------------------------

// A 64 x 64 tile of A B^T in float32: element (m, k) of A is at a[m am + k ak].
template <class T>
struct Operand {
    const T* p;
    int64_t outer, inner;  // strides of the tile's and of the summed dimension
    int64_t size;          // of the tile's dimension
};
constexpr int kTile = 64, kDepth = 16;

template <class T>
__device__ __forceinline__ void tile_product(const Operand<T>& a, const Operand<T>& b, int64_t depth, int64_t m0, int64_t n0,
                                             float (&acc)[4][4]) {
    __shared__ float sa[kDepth][kTile + 4], sb[kDepth][kTile + 4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    const int tm = threadIdx.x / 16 * 4, tn = threadIdx.x % 16 * 4;
    for (int64_t k0 = 0; k0 < depth; k0 += kDepth) {
        __syncthreads();
        for (int i = threadIdx.x; i < kTile * kDepth; i += kThreads) {
            const int m = i / kDepth, k = i % kDepth;
            const bool in = k0 + k < depth;
            sa[k][m] = in && m0 + m < a.size ? to_float(a.p[(m0 + m) * a.outer + (k0 + k) * a.inner]) : 0.0f;
            sb[k][m] = in && n0 + m < b.size ? to_float(b.p[(n0 + m) * b.outer + (k0 + k) * b.inner]) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDepth; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][tm + i], sb[k][tn + j], acc[i][j]);
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) stats_kernel(Ws w, Operand<T> hidden, Operand<T> weight, int cols, float scale) {
    pdl_enter();
    const int64_t count = w.head->count, m0 = static_cast<int64_t>(blockIdx.y) * kTile, n0 = static_cast<int64_t>(blockIdx.x) * kTile;
    if (m0 >= count) return;
    float acc[4][4];
    tile_product(hidden, weight, cols, m0, n0, acc);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = m0 + threadIdx.x / 16 * 4 + i;
        const int label = r < count ? w.labels[r] : -1;
        MaxSum s{-INFINITY, 0.0f};
        float z[4];
        bool nan = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + threadIdx.x % 16 * 4 + j;
            z[j] = n < weight.size ? acc[i][j] * scale : -INFINITY;
            if (n == label) w.picked[r] = z[j];
            nan |= z[j] != z[j];
            s.m = fmaxf(s.m, z[j]);
        }
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) s.m = fmaxf(s.m, __shfl_xor_sync(kFull, s.m, o));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (s.m != -INFINITY) s.s += ex2(z[j] - s.m);
        if (nan) s.s = NAN;
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) s.s += __shfl_xor_sync(kFull, s.s, o);
        if (threadIdx.x % 16 == 0 && r < count) w.parts[blockIdx.x * w.rows_pad + r] = make_float2(s.m, s.s);
    }
}

__global__ void __launch_bounds__(kThreads) join_kernel(LossArgs a, Ws w, int64_t parts) {
    pdl_enter();
    const int64_t count = w.head->count;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; r < count; r += static_cast<int64_t>(gridDim.x) * kThreads) {
        float m = -INFINITY, s = 0.0f;
        for (int64_t i = 0; i < parts; ++i) {
            const float2 p = w.parts[i * w.rows_pad + r];
            const float n = fmaxf(m, p.x);
            if (n != -INFINITY) s = s * ex2(m - n) + p.y * ex2(p.x - n);
            else s += p.y;
            m = n;
        }
        const float log = logf(s);
        const int label = w.labels[r], to = w.map[r];
        const float lse = fmaf(m, kLN2, log);
        a.losses[to] = label >= 0 ? fmaf(m - w.picked[r], kLN2, log) : lse;
        if (a.lse) a.lse[to] = lse;
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) probs_kernel(Ws w, Operand<T> hidden, Operand<T> weight, int cols, float scale, int64_t first,
                                                         T* probs, int64_t piece) {
    pdl_enter();
    const int64_t count = w.head->count, m0 = static_cast<int64_t>(blockIdx.y) * kTile, n0 = static_cast<int64_t>(blockIdx.x) * kTile;
    if (m0 >= (count + kTileRows - 1) / kTileRows * kTileRows) return;
    float acc[4][4];
    tile_product(hidden, weight, cols, m0, n0, acc);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = m0 + threadIdx.x / 16 * 4 + i;
        const bool in = r < count;
        const float s = w.head->scale, lse = in ? w.lse[r] : 0.0f, c = in ? w.coef[r] * s : 0.0f, o = in ? w.onehot[r] * s : 0.0f;
        const int64_t label = in ? w.labels[r] - first : -1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + threadIdx.x % 16 * 4 + j;
            float v = c * ex2(fmaf(acc[i][j], scale, -lse));
            if (n == label && w.labels[r] >= 0) v -= o;
            probs[r * piece + n] = from_float<T>(in && n < weight.size ? v : 0.0f);
        }
    }
}

// sums (+)= a b^T
template <class T>
__global__ void __launch_bounds__(kThreads) dhidden_kernel(Ws w, Operand<T> a, Operand<T> b, int64_t depth, int64_t pitch, int first) {
    pdl_enter();
    const int64_t count = w.head->count, m0 = static_cast<int64_t>(blockIdx.y) * kTile, n0 = static_cast<int64_t>(blockIdx.x) * kTile;
    if (m0 >= count) return;
    float acc[4][4];
    tile_product(a, b, depth, m0, n0, acc);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t r = m0 + threadIdx.x / 16 * 4 + i, c = n0 + threadIdx.x % 16 * 4 + j;
            if (r >= count || c >= b.size) continue;
            float* p = w.sums + r * pitch + c;
            *p = first ? acc[i][j] : *p + acc[i][j];
        }
}
template <class T>
__global__ void __launch_bounds__(kThreads) emit_kernel(LossArgs a, Ws w, int64_t pitch) {
    pdl_enter();
    const int64_t n = w.head->count * a.cols;
    const float u = w.head->unscale;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t r = i / a.cols, c = i - r * a.cols;
        static_cast<T*>(a.dhidden)[static_cast<int64_t>(w.map[r]) * a.cols + c] = from_float<T>(u * w.sums[r * pitch + c]);
    }
}
template <class T>
__global__ void __launch_bounds__(kThreads) dweight_kernel(Ws w, Operand<T> a, Operand<T> b, T* dweight) {
    pdl_enter();
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTile, n0 = static_cast<int64_t>(blockIdx.x) * kTile;
    float acc[4][4];
    tile_product(a, b, w.head->count, m0, n0, acc);
    const float u = w.head->unscale;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t r = m0 + threadIdx.x / 16 * 4 + i, c = n0 + threadIdx.x % 16 * 4 + j;
            if (r < a.size && c < b.size) dweight[r * b.size + c] = from_float<T>(u * acc[i][j]);
        }
}

Ws workspace(const LossArgs& a, const LossPlan& p) {
    auto f = [&](size_t at) { return reinterpret_cast<float*>(a.ws + at); };
    return Ws{reinterpret_cast<LossHead*>(a.ws + p.head), reinterpret_cast<int*>(a.ws + p.map), reinterpret_cast<int*>(a.ws + p.labels),
              f(p.lse), f(p.coef), f(p.onehot), reinterpret_cast<float2*>(a.ws + p.parts_at), f(p.picked), f(p.sums), p.rows_pad};
}

template <class T>
struct Packed {
    T* hidden;
    const T* weight;
    int64_t pitch;
};

template <class T>
cudaError_t pack(const LossArgs& a, const LossPlan& p, const Ws& w, int backward, Packed<T>* out, cudaStream_t stream) {
    out->hidden = reinterpret_cast<T*>(a.ws + p.hidden);
    out->weight = static_cast<const T*>(a.weight);
    out->pitch = p.pitch;
    cudaError_t e = launch_dependent(rows_kernel, dim3(1), kScanThreads, 0, 1, stream, a, w, backward);
    if (e != cudaSuccess) return e;
    auto ctas = [](int64_t rows) { return dim3(static_cast<unsigned>(std::min<int64_t>(ceil_div(rows, kThreads / 32), 1 << 16))); };
    e = launch_dependent(pack_kernel<T>, ctas(p.rows_pad), kThreads, 0, 1, stream, a, w, static_cast<const T*>(a.hidden), a.rows,
                         out->hidden, p.pitch, p.rows_pad, backward ? static_cast<T*>(a.dhidden) : nullptr);
    if (e != cudaSuccess || !p.pack_weight) return e;
    T* to = reinterpret_cast<T*>(a.ws + p.weight);
    out->weight = to;
    Ws all{};
    return launch_dependent(pack_kernel<T>, ctas(a.vocab), kThreads, 0, 1, stream, a, all, static_cast<const T*>(a.weight), a.vocab,
                            to, p.pitch, a.vocab, nullptr);
}

template <class T>
cudaError_t forward(const LossArgs& a, cudaStream_t stream) {
    const LossPlan p(a.rows, a.cols, a.vocab, false);
    const Ws w = workspace(a, p);
    Packed<T> k;
    cudaError_t e = pack(a, p, w, 0, &k, stream);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(p.parts), static_cast<unsigned>(p.rows_pad / kTile));
    e = launch_dependent(stats_kernel<T>, grid, kThreads, 0, 1, stream, w, Operand<T>{k.hidden, k.pitch, 1, p.rows_pad},
                         Operand<T>{k.weight, k.pitch, 1, a.vocab}, a.cols, a.logit_scale * kL2E);
    if (e != cudaSuccess) return e;
    return launch_dependent(join_kernel, dim3(static_cast<unsigned>(ceil_div(a.rows, kThreads))), kThreads, 0, 1, stream, a, w, p.parts);
}

template <class T>
cudaError_t backward(const LossArgs& a, cudaStream_t stream) {
    const LossPlan p(a.rows, a.cols, a.vocab, true);
    const Ws w = workspace(a, p);
    Packed<T> k;
    cudaError_t e = pack(a, p, w, 1, &k, stream);
    T* probs = reinterpret_cast<T*>(a.ws + p.probs);
    const unsigned tiles = static_cast<unsigned>(p.rows_pad / kTile), col_tiles = static_cast<unsigned>(ceil_div(a.cols, kTile));
    for (int64_t first = 0; first < a.vocab && e == cudaSuccess; first += p.piece) {
        const int64_t n = std::min(p.piece, a.vocab - first);
        const T* weight = k.weight + first * k.pitch;
        const unsigned across = static_cast<unsigned>(ceil_div(n, kTile));
        e = launch_dependent(probs_kernel<T>, dim3(across, tiles), kThreads, 0, 1, stream, w, Operand<T>{k.hidden, k.pitch, 1, p.rows_pad},
                             Operand<T>{weight, k.pitch, 1, n}, a.cols, a.logit_scale * kL2E, first, probs, p.piece);
        if (e == cudaSuccess && a.dhidden)
            e = launch_dependent(dhidden_kernel<T>, dim3(col_tiles, tiles), kThreads, 0, 1, stream, w,
                                 Operand<T>{probs, p.piece, 1, p.rows_pad}, Operand<T>{weight, 1, k.pitch, a.cols}, n, p.pitch,
                                 first == 0 ? 1 : 0);
        if (e == cudaSuccess && a.dweight)
            e = launch_dependent(dweight_kernel<T>, dim3(col_tiles, across), kThreads, 0, 1, stream, w, Operand<T>{probs, 1, p.piece, n},
                                 Operand<T>{k.hidden, 1, k.pitch, a.cols}, static_cast<T*>(a.dweight) + first * a.cols);
    }
    if (e != cudaSuccess || !a.dhidden) return e;
    const int64_t ctas = std::min<int64_t>(ceil_div(a.rows * a.cols, kThreads), 1 << 16);
    return launch_dependent(emit_kernel<T>, dim3(static_cast<unsigned>(ctas)), kThreads, 0, 1, stream, a, w, p.pitch);
}

}  // namespace loss

cudaError_t launch_loss(int dtype, const LossArgs& a, cudaStream_t stream) {
    return dtype == TR_BF16 ? loss::forward<__nv_bfloat16>(a, stream) : loss::forward<__half>(a, stream);
}
cudaError_t launch_loss_backward(int dtype, const LossArgs& a, cudaStream_t stream) {
    return dtype == TR_BF16 ? loss::backward<__nv_bfloat16>(a, stream) : loss::backward<__half>(a, stream);
}

}  // namespace tr
