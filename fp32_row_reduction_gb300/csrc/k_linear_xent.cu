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
#include "tr_mma.cuh"
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
    width = grad_width = mma::kMaxWidth;
    splits = 1;
    parts = 2 * ceil_div(vocab, width);
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
        sums = take(splits * rows_pad * pitch * 4);
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

template <class T>
constexpr uint32_t kTypeBits = 0;
template <>
constexpr uint32_t kTypeBits<__nv_bfloat16> = 1;

// What the four products share. `first`: the piece of the vocabulary begins there and has `n` words.
struct Product {
    Ws w;
    mma::Limits lim;
    int cols, splits, width;
    int64_t first, n;
    float scale;      // log2(e) logit_scale
    void* to;         // probs, dhidden or dweight
    int64_t pitch;    // of its rows (of `sums` for the hidden gradient)
    int begun, last;  // hidden gradient: whether the sums have earlier pieces, and whether this one completes them
    int wide;         // rows of `to` start on 16 bytes
};

__device__ __forceinline__ int tiles_of(int64_t n, int size) { return static_cast<int>((n + size - 1) / size); }

template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// 32 columns from c on of a row per lane (null: none), of which those below `cols` are written, rounded to T. Rows that start on 16
// bytes take 16-byte stores; others are turned in shared memory, so that a warp writes 32 columns of one row at a time.
template <class T>
__device__ __forceinline__ void store_columns(T* row, int c, int cols, const float (&v)[32], bool wide, float* turn) {
    if (wide) {
        if (!row) return;
#pragma unroll
        for (int g = 0; g < 4; ++g)
            if (c + 8 * g < cols)
                *reinterpret_cast<uint4*>(row + c + 8 * g) = make_uint4(pack2<T>(v[8 * g], v[8 * g + 1]), pack2<T>(v[8 * g + 2], v[8 * g + 3]),
                                                                        pack2<T>(v[8 * g + 4], v[8 * g + 5]), pack2<T>(v[8 * g + 6], v[8 * g + 7]));
        return;
    }
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 32; ++i) turn[lane * 33 + i] = v[i];
    __syncwarp();
    const unsigned long long mine = reinterpret_cast<unsigned long long>(row);
    for (int i = 0; i < 32; ++i) {
        T* p = reinterpret_cast<T*>(__shfl_sync(kFull, mine, i));
        if (p && c + lane < cols) p[c + lane] = from_float<T>(turn[i * 33 + lane]);
    }
}

__device__ __forceinline__ void spoil(float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = NAN;
}

// Forward: (maximum, sum of 2^(z - maximum)) of each half of a tile's columns, and the label's z.
template <class T>
__global__ void __cluster_dims__(2) __launch_bounds__(mma::kThreads, 1)
    stats_kernel(const __grid_constant__ CUtensorMap hidden, const __grid_constant__ CUtensorMap weight, const __grid_constant__ Product p) {
    int64_t count = 0;
    mma::run<false, false>(
        &hidden, &weight, kTypeBits<T>, p.lim,
        [&] {
            count = p.w.head->count;
            return mma::Work{tiles_of(count, kTileRows), tiles_of(p.n, p.width), 1, tiles_of(p.cols, mma::kDepth), p.width};
        },
        [&](const mma::Unit& u, int row, int half, int first, int last, uint32_t at, bool ok, float*) {
            const int limit = static_cast<int>(min(static_cast<int64_t>(last), p.n - u.n));  // columns of the vocabulary
            const int label = row < count ? p.w.labels[row] - u.n : -1;
            float m = -INFINITY, s = 0.0f;
            for (int c = first; c < limit; c += 32) {
                float z[32];
                mma::load_columns(at + c, z);
                if (!ok) spoil(z);
#pragma unroll
                for (int i = 0; i < 32; ++i) z[i] *= p.scale;
                if (label >= c && label < min(c + 32, limit)) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (label == c + i) p.w.picked[row] = z[i];
                }
                if (c + 32 > limit) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c + i >= limit) z[i] = -INFINITY;
                }
                float top = z[0];
#pragma unroll
                for (int i = 1; i < 32; ++i) top = fmaxf(top, z[i]);
                const float most = fmaxf(m, top), from = most == -INFINITY ? 0.0f : most;
                float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < 32; ++i) part[i & 3] += ex2(z[i] - from);
                s = fmaf(s, ex2(m - from), (part[0] + part[1]) + (part[2] + part[3]));
                m = most;
            }
            if (row < count) p.w.parts[(2 * static_cast<int64_t>(u.n / p.width) + half) * p.w.rows_pad + row] = make_float2(m, s);
        });
}

// Backward: scale dz / logit_scale of a piece, rounded. Rows and words beyond the last are zeros up to the tile's end.
template <class T>
__global__ void __cluster_dims__(2) __launch_bounds__(mma::kThreads, 1)
    probs_kernel(const __grid_constant__ CUtensorMap hidden, const __grid_constant__ CUtensorMap weight, const __grid_constant__ Product p) {
    int64_t count = 0;
    float times = 0.0f;
    mma::run<false, false>(
        &hidden, &weight, kTypeBits<T>, p.lim,
        [&] {
            count = p.w.head->count;
            times = p.w.head->scale;
            return mma::Work{tiles_of(count, kTileRows), tiles_of(p.n, p.width), 1, tiles_of(p.cols, mma::kDepth), p.width};
        },
        [&](const mma::Unit& u, int row, int, int first, int last, uint32_t at, bool ok, float* turn) {
            const bool in = row < count;
            const int limit = static_cast<int>(min(static_cast<int64_t>(last), p.n - u.n));
            const float lse = in ? p.w.lse[row] : 0.0f, coef = in ? p.w.coef[row] * times : 0.0f;
            const float onehot = in ? p.w.onehot[row] * times : 0.0f;
            const int word = in ? p.w.labels[row] : -1;
            const int label = word >= 0 ? static_cast<int>(word - p.first) - u.n : -1;
            T* to = static_cast<T*>(p.to) + row * p.pitch + u.n;
            for (int c = first; c < last; c += 32) {
                float z[32];
                mma::load_columns(at + c, z);
                if (!ok) spoil(z);
#pragma unroll
                for (int i = 0; i < 32; ++i) z[i] = coef * ex2(fmaf(z[i], p.scale, -lse));
                if (label >= c && label < c + 32) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (label == c + i) z[i] -= onehot;
                }
                if (!in || c + 32 > limit) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!in || c + i >= limit) z[i] = 0.0f;
                }
                store_columns<T>(to, c, last, z, true, turn);
            }
        });
}

// Backward: the piece's part of the hidden gradient, added to those of earlier pieces; the last one writes the gradient.
template <class T>
__global__ void __cluster_dims__(2) __launch_bounds__(mma::kThreads, 1)
    dhidden_kernel(const __grid_constant__ CUtensorMap probs, const __grid_constant__ CUtensorMap weight, const __grid_constant__ Product p) {
    int64_t count = 0;
    float times = 0.0f;
    mma::run<false, true>(
        &probs, &weight, kTypeBits<T>, p.lim,
        [&] {
            count = p.w.head->count;
            times = p.w.head->unscale;
            return mma::Work{tiles_of(count, kTileRows), tiles_of(p.cols, p.width), p.splits, tiles_of(p.n, mma::kDepth), p.width};
        },
        [&](const mma::Unit& u, int row, int, int first, int last, uint32_t at, bool ok, float* turn) {
            const bool in = row < count;
            float* sums = p.w.sums + (u.split * p.w.rows_pad + row) * p.pitch + u.n;
            T* to = in && p.last ? static_cast<T*>(p.to) + static_cast<int64_t>(p.w.map[row]) * p.cols + u.n : nullptr;
            const int cols = static_cast<int>(min(static_cast<int64_t>(last), p.pitch - u.n));
            for (int c = first; c < cols; c += 32) {
                float z[32];
                mma::load_columns(at + c, z);
                if (!ok) spoil(z);
                if (u.begin == u.end) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) z[i] = 0.0f;
                }
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    if (!in || c + 4 * g >= cols) continue;
                    float4* q = reinterpret_cast<float4*>(sums + c) + g;
                    if (p.begun) {
                        const float4 f = *q;
                        z[4 * g] += f.x;
                        z[4 * g + 1] += f.y;
                        z[4 * g + 2] += f.z;
                        z[4 * g + 3] += f.w;
                    }
                    if (!p.last) *q = make_float4(z[4 * g], z[4 * g + 1], z[4 * g + 2], z[4 * g + 3]);
                }
                if (p.last) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) z[i] *= times;
                    store_columns<T>(to, c, min(last, p.cols - u.n), z, p.wide, turn);
                }
            }
        });
}

// Backward: the piece's rows of the weight's gradient.
template <class T>
__global__ void __cluster_dims__(2) __launch_bounds__(mma::kThreads, 1)
    dweight_kernel(const __grid_constant__ CUtensorMap probs, const __grid_constant__ CUtensorMap hidden, const __grid_constant__ Product p) {
    float times = 0.0f;
    mma::run<true, true>(
        &probs, &hidden, kTypeBits<T>, p.lim,
        [&] {
            times = p.w.head->unscale;
            return mma::Work{tiles_of(p.n, kTileRows), tiles_of(p.cols, p.width), 1, tiles_of(p.w.head->count, mma::kDepth), p.width};
        },
        [&](const mma::Unit& u, int row, int, int first, int last, uint32_t at, bool ok, float* turn) {
            T* to = row < p.n ? static_cast<T*>(p.to) + (p.first + row) * p.cols + u.n : nullptr;
            const int cols = min(last, p.cols - u.n);
            for (int c = first; c < cols; c += 32) {
                float z[32];
                mma::load_columns(at + c, z);
                if (!ok) spoil(z);
#pragma unroll
                for (int i = 0; i < 32; ++i) z[i] = u.begin == u.end ? 0.0f : z[i] * times;
                store_columns<T>(to, c, cols, z, p.wide, turn);
            }
        });
}

// The parts of a hidden gradient whose depth was split, added in order.
template <class T>
__global__ void __launch_bounds__(kThreads) emit_kernel(LossArgs a, Ws w, int64_t pitch, int splits) {
    pdl_enter();
    const int64_t n = w.head->count * a.cols;
    const float u = w.head->unscale;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t r = i / a.cols, c = i - r * a.cols;
        float s = 0.0f;
        for (int k = 0; k < splits; ++k) s += w.sums[(k * w.rows_pad + r) * pitch + c];
        static_cast<T*>(a.dhidden)[static_cast<int64_t>(w.map[r]) * a.cols + c] = from_float<T>(u * s);
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

// ---- launches -------------------------------------------------------------------------

// A tensor map of rows x cols elements (rows `pitch` apart) in boxes of 64 columns.
using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                            const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
Encode encoder() {
    static const Encode fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<Encode>(p);
    }();
    return fn;
}
template <class T>
cudaError_t map_of(CUtensorMap* map, const T* p, int64_t rows, int64_t cols, int64_t pitch, int box_rows) {
    const Encode encode = encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t size[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)}, stride[1] = {static_cast<cuuint64_t>(pitch) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)}, step[2] = {1, 1};
    const CUresult r = encode(map, kTypeBits<T> ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<T*>(p), size,
                              stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// CTA pairs for `units` of work.
template <class K>
cudaError_t launch_product(K kernel, const CUtensorMap& a, const CUtensorMap& b, const Product& p, int64_t units, cudaStream_t stream) {
    const int resident = resident_ctas(reinterpret_cast<const void*>(kernel), mma::kThreads, mma::kSmem, 2);
    if (resident < 2) return cudaErrorInvalidConfiguration;
    const int64_t pairs = std::min<int64_t>(units, resident / 2);
    return launch_dependent(kernel, dim3(static_cast<unsigned>(2 * pairs)), mma::kThreads, mma::kSmem, 1, stream, a, b, p);
}

template <class T>
cudaError_t forward(const LossArgs& a, cudaStream_t stream) {
    const LossPlan p(a.rows, a.cols, a.vocab, false);
    const Ws w = workspace(a, p);
    Packed<T> k;
    cudaError_t e = pack(a, p, w, 0, &k, stream);
    CUtensorMap hidden, weight;
    if (e == cudaSuccess) e = map_of(&hidden, k.hidden, p.rows_pad, a.cols, k.pitch, mma::kRows);
    if (e == cudaSuccess) e = map_of(&weight, k.weight, a.vocab, a.cols, k.pitch, p.width / 2);
    if (e != cudaSuccess) return e;
    Product d{};
    d.w = w;
    d.lim = mma::Limits{device_error_word(), debug_flags_now()};
    d.cols = a.cols;
    d.width = p.width;
    d.n = a.vocab;
    d.scale = a.logit_scale * kL2E;
    e = launch_product(stats_kernel<T>, hidden, weight, d, p.rows_pad / kTileRows * ceil_div(a.vocab, p.width), stream);
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
    CUtensorMap hidden_rows, hidden_cols, probs_rows, probs_cols;
    if (e == cudaSuccess) e = map_of(&hidden_rows, k.hidden, p.rows_pad, a.cols, k.pitch, mma::kRows);
    if (e == cudaSuccess) e = map_of(&hidden_cols, k.hidden, p.rows_pad, a.cols, k.pitch, mma::kDepth);
    if (e == cudaSuccess) e = map_of(&probs_rows, probs, p.rows_pad, p.piece, p.piece, mma::kRows);
    if (e == cudaSuccess) e = map_of(&probs_cols, probs, p.rows_pad, p.piece, p.piece, mma::kDepth);
    const bool align = a.cols % 8 == 0;
    const int64_t row_tiles = p.rows_pad / kTileRows;
    for (int64_t first = 0; first < a.vocab && e == cudaSuccess; first += p.piece) {
        const int64_t n = std::min(p.piece, a.vocab - first);
        CUtensorMap weight_rows, weight_cols;
        e = map_of(&weight_rows, k.weight + first * k.pitch, n, a.cols, k.pitch, p.width / 2);
        if (e == cudaSuccess) e = map_of(&weight_cols, k.weight + first * k.pitch, n, a.cols, k.pitch, mma::kDepth);
        if (e != cudaSuccess) break;
        Product d{};
        d.w = w;
        d.lim = mma::Limits{device_error_word(), debug_flags_now()};
        d.cols = a.cols;
        d.first = first;
        d.n = n;
        d.scale = a.logit_scale * kL2E;
        d.width = p.width;
        d.to = probs;
        d.pitch = p.piece;
        e = launch_product(probs_kernel<T>, hidden_rows, weight_rows, d, row_tiles * ceil_div(n, p.width), stream);
        if (e == cudaSuccess && a.dhidden) {
            d.width = p.grad_width;
            d.to = a.dhidden;
            d.pitch = p.pitch;
            d.begun = first > 0;
            d.last = p.splits == 1 && first + n == a.vocab;
            d.splits = p.splits;
            d.wide = align && reinterpret_cast<uintptr_t>(a.dhidden) % 16 == 0;
            e = launch_product(dhidden_kernel<T>, probs_rows, weight_cols, d, row_tiles * ceil_div(a.cols, d.width) * p.splits, stream);
        }
        if (e == cudaSuccess && a.dweight) {
            d.width = p.grad_width;
            d.to = a.dweight;
            d.wide = align && reinterpret_cast<uintptr_t>(a.dweight) % 16 == 0;
            e = launch_product(dweight_kernel<T>, probs_cols, hidden_cols, d, ceil_div(n, kTileRows) * ceil_div(a.cols, d.width), stream);
        }
    }
    if (e != cudaSuccess || !a.dhidden || p.splits == 1) return e;
    const int64_t ctas = std::min<int64_t>(ceil_div(a.rows * a.cols, kThreads), 1 << 16);
    return launch_dependent(emit_kernel<T>, dim3(static_cast<unsigned>(ctas)), kThreads, 0, 1, stream, a, w, p.pitch, p.splits);
}

}  // namespace loss

cudaError_t launch_loss(int dtype, const LossArgs& a, cudaStream_t stream) {
    return dtype == TR_BF16 ? loss::forward<__nv_bfloat16>(a, stream) : loss::forward<__half>(a, stream);
}
cudaError_t launch_loss_backward(int dtype, const LossArgs& a, cudaStream_t stream) {
    return dtype == TR_BF16 ? loss::backward<__nv_bfloat16>(a, stream) : loss::backward<__half>(a, stream);
}

}  // namespace tr
