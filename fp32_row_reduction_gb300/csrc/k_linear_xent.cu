// Softmax cross entropy of logits = logit_scale hidden weight^T that are never kept, and its gradients.
//
// With z = log2(e) logits, forward: every row's maximum m and sum of 2^(z - m) over half of each tile of the vocabulary (up to 128
// words), which a last kernel joins: lse = ln 2 (m + log2 sum), loss = ln 2 (m - z_label) + ln sum, so that the loss of a certain row
// is no difference of large numbers. Backward, for one piece of the vocabulary after another:
// dz = (dloss + dlse) 2^(z - lse) - dloss [label], rounded to the inputs' type for the products dhidden += dz weight
// (in float32 over the pieces) and dweight = dz^T hidden. The rounding is one of T's half steps of each dz, relative to a dz that has
// the label's -1 in it already; it adds as much as a third to the outputs' error (bf16 201 x 320 x 136: 2.2e-3 instead of 1.7e-3). Where the products are
// short, dz is taken in two terms of T, the second what the first one's rounding left, and nothing is added. That costs
// 2 to 8 us (37 x 1537 x 5003 f16 47.5 us instead of 44.7); for 8192 x 4096 x 50257 it would be 9.5 ms instead of 5.5.
//
// Rows that have a loss are packed first: the products do no work for the others, and what those hold, which may be no
// number, is not read as the depth of the weight's gradient.
//
// Bound by the tensor cores, and at length by power: 8192 x 4096 x 50257 bf16 with 10% of the rows ignored, forward 1.55 ms at 1.9 GHz
// (1960 TFLOP/s) and 1.70 ms call after call at 1.5 GHz and 1370 W; gradients 4.9 and 5.5 ms (1860 and 1660). Few rows are bound
// by reading the weight: 48 x 5120 f16 forward 88 us (5.8 TB/s).
#include <algorithm>
#include <cmath>

#include "tr_launch.h"
#include "tr_mma.cuh"
#include "tr_vocab.cuh"
#include "tr_vocab.h"

namespace tr {

constexpr int kPairs = 76;  // CTA pairs of the GPU that the plan is made for
// Blocks of the depth (the piece's words, or the rows) that the gradients are summed over in tensor memory, which rounds toward zero: 131072
// words in one sum came out 2.5e-4 too small, as much as float16's last rounding; parts of 8192 are 2e-5. The parts of longer depths
// are added in registers by a kernel of its own (8192 x 4096 x 50257 takes 1.3% longer in parts, 3% in
// parts of 4096; the registers would cost 64 x 2047 x 30000, whose depths are one part each, 215 us instead of 178).
constexpr int kGradPart = 128;
// And of the logits (blocks of the width): sums of 1024 are off by 1e-7 to 3e-7 of the losses, where binary32 products rounded to nearest are off by 1e-7,
// and by 1e-6 of the small losses of a few likely words. Where no pair has more than one tile they are of 512, for 2% at most; a
// training batch would take 10% longer, 48 x 5120 x 50257 7%. (Sums of 256: 48 x 5120 140 us instead of 91: a thread's 128 columns of a part take 4000 cycles.)
constexpr int kLogitPart = 16, kShortLogitPart = 8;

LossPlan::LossPlan(int64_t rows, int64_t cols, int64_t vocab, bool backward) {
    size_t at = 0;
    auto take = [&](int64_t n) {
        const size_t here = at;
        at += (static_cast<size_t>(n) + 255) / 256 * 256;
        return here;
    };
    rows_pad = round_up(rows, kTileRows);
    pitch = round_up(cols, 8);
    pack_weight = cols % 8 != 0;
    const int64_t row_tiles = rows_pad / kTileRows, words = round_up(vocab, 256);
    grad_width = cols > 128 ? mma::kMaxWidth : 128;  // (half as wide a tile takes half as long)
    const int64_t across = ceil_div(cols, grad_width);
    const int64_t hidden_tiles = row_tiles * across, weight_tiles = words / kTileRows * across;
    // Few tiles of the hidden gradient have their depth, the words, split over the pairs.
    const auto split_depth = [&](int64_t n) { return std::max<int64_t>(1, std::min(kPairs / hidden_tiles, n / (4 * mma::kDepth))); };
    // dz in two terms, where the second takes a pair no more than kFineBlocks (4 us), or where writing a tile out takes longer than its products
    // anyway: kFineDepth blocks, 128 rows or words (32 x 4096 x 50257: 286 us instead of 280; 256 x 2048 x 32000 would take 140 instead of 129).
    constexpr int64_t kFineBlocks = 16, kFineDepth = 2;
    const int64_t split_words = split_depth(words);
    fine_hidden = vocab <= kFineDepth * mma::kDepth || ceil_div(hidden_tiles * split_words, kPairs) * ceil_div(words / mma::kDepth, split_words) <= kFineBlocks;
    fine_weight = rows <= kFineDepth * mma::kDepth || ceil_div(weight_tiles, kPairs) * (rows_pad / mma::kDepth) <= kFineBlocks;
    terms = fine_hidden || fine_weight ? 2 : 1;
    // dz of a piece: 2^27 values (256 MB), and at least 4096 columns, so that the sums over the pieces cost little
    constexpr int64_t kValues = int64_t{1} << 27, kLeast = 4096;
    const int64_t most = std::max(kLeast, kValues / (rows_pad * terms) / 256 * 256);
    const int64_t pieces = ceil_div(vocab, std::min(most, words));
    piece = round_up(ceil_div(vocab, pieces), 256);
    // The width whose tiles come out even over the pairs of a GPU's CTAs. A narrow tile reads the rows of hidden more often (the
    // 24), which a single tile of rows does not feel in the forward pass: there a narrower tile only splits the weight's reading more
    // evenly. Backward, the tiles fill whole multiples of 256 words.
    width = mma::kMaxWidth;
    constexpr int kRead = 24;
    int64_t least = INT64_MAX;
    for (int n = mma::kMaxWidth; n >= 64; n = backward ? n / 2 : n - 32) {
        const int64_t cost = ceil_div(row_tiles * ceil_div(backward ? piece : vocab, n), kPairs) * (n + (backward || row_tiles > 1 ? kRead : 0));
        if (cost < least) least = cost, width = n;
    }
    // A single tile of rows has the hidden gradient's depth split into no longer parts than are summed at once: its weight's tiles, bound by their writing,
    // would feel the kernel that adds parts in registers (32 x 4096 x 50257: 296 us instead of 280; for 1024 x 1024 x 50257 that kernel
    // is the better one, 236 instead of 244).
    const int64_t hidden_blocks = piece / mma::kDepth * (fine_hidden ? 2 : 1), weight_blocks = rows_pad / mma::kDepth * (fine_weight ? 2 : 1);
    splits = static_cast<int>(split_depth(piece));
    if (splits > 1 && row_tiles == 1) splits = static_cast<int>(std::max<int64_t>(splits, ceil_div(hidden_blocks, kGradPart)));
    parted = std::max(ceil_div(hidden_blocks, splits), weight_blocks) > kGradPart;
    logit_part = row_tiles * (words / 256) <= kPairs ? kShortLogitPart : kLogitPart;
    parts = 2 * ceil_div(vocab, width);
    head = take(sizeof(LossHead));
    map = take(rows_pad * 4);
    labels = take(rows_pad * 4);
    hidden = take(rows_pad * pitch * 2);
    weight = pack_weight ? take(vocab * pitch * 2) : at;
    lse = coef = onehot = probs = sums = parts_at = picked = at;
    // Fewer rows have longer pieces, more splits or narrower tiles, so that they may use more of what follows. It is as large as any call of no more
    // rows needs it: a workspace for the longest batch is one for all shorter ones.
    if (backward) {
        lse = take(rows_pad * 4);
        coef = take(rows_pad * 4);
        onehot = take(rows_pad * 4);
        // Two terms take hidden_tiles or weight_tiles times their depth <= kFineBlocks kPairs blocks, or they are of a single tile of rows, or of words.
        // Tiles of rows times terms, `dz`, are times 256 and a piece <= min(words, max(kLeast, kValues / that)).
        const int64_t fine_tiles = vocab <= kFineDepth * mma::kDepth ? row_tiles : std::max<int64_t>(1, kFineBlocks * kPairs * mma::kDepth / (across * words));
        const int64_t dz = std::max(row_tiles, 2 * std::min(row_tiles, fine_tiles));
        probs = take(2 * std::min(kTileRows * dz * words, std::max(kTileRows * dz * kLeast, kValues)));
        // splits row_tiles, in tiles: with no more than `split` tiles of rows the depth is split, into at most words / 256 parts, and no more than fill
        // the pairs or (a single tile of rows) than there are parts of kGradPart in two terms
        const int64_t split = std::min(row_tiles, kPairs / 2 / across);
        const int64_t tiles = std::min(split * (words / 256), std::max(kPairs / across, ceil_div(2 * words, kGradPart * mma::kDepth)));
        sums = take(4 * pitch * kTileRows * std::max({splits * row_tiles, row_tiles, tiles}));
    } else {
        // A width n is taken only where ceil(row_tiles t(n) / kPairs) (n + kRead) <= that of every other m, t the tiles across, for which
        // row_tiles (t(n) (n + kRead) - t(m) (m + kRead)) < kPairs (m + kRead) has to hold; or for a single tile of rows.
        int64_t tiles = 0;
        for (int n = 64; n <= mma::kMaxWidth; n += 32) {
            int64_t last = row_tiles;
            for (int m = 64; m <= mma::kMaxWidth; m += 32) {
                const int64_t more = ceil_div(vocab, n) * (n + kRead) - ceil_div(vocab, m) * (m + kRead);
                if (more > 0) last = std::min(last, (kPairs * (m + kRead) - 1) / more);
            }
            tiles = std::max(tiles, ceil_div(vocab, n) * std::max<int64_t>(last, 1));
        }
        parts_at = take(16 * kTileRows * std::max(tiles, parts / 2 * row_tiles));
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

// A CTA lists them in order (map[i]: the i-th one's row) and, with `write`, in the workspace, with their labels (-1: outside the vocabulary)
// and, backward, their coefficients: of the probability (dloss + dlse) and of the label (dloss); the outputs of rows without a loss
// are zeros then. ITEMS: rows of a thread at a time, 32 apart. All threads get the count.
template <int ITEMS>
__device__ __forceinline__ int64_t list_rows(const LossArgs& a, const Ws& w, int backward, bool write, int* map) {
    __shared__ int warp_count[32];
    __shared__ float warp_most[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned before = (1u << lane) - 1u;
    int64_t count = 0;
    float most = 0.0f, most_d = 0.0f;
    for (int64_t r0 = 0; r0 < a.rows; r0 += ITEMS * kScanThreads) {
        const int64_t r1 = r0 + warp * (32 * ITEMS) + lane;
        int64_t label[ITEMS];
        float lse[ITEMS], d[ITEMS], e[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int64_t r = r1 + 32 * i;
            const bool in = r < a.rows;
            label[i] = in ? a.labels[r] : a.ignore;
            if (write && backward) {
                lse[i] = in ? a.lse_in[r] : 0.0f;
                d[i] = in && a.dloss ? a.dloss[r] : 1.0f;
                e[i] = in && a.dlse ? a.dlse[r] : 0.0f;
            }
        }
        unsigned votes[ITEMS];
        int total = 0;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            votes[i] = __ballot_sync(kFull, label[i] != a.ignore);
            total += __popc(votes[i]);
        }
        __syncthreads();
        if (lane == 0) warp_count[warp] = total;
        __syncthreads();
        const int mine = warp_count[lane];
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += v;
        }
        int64_t at = count + __shfl_sync(kFull, inc - mine, warp);
        count += __shfl_sync(kFull, inc, 31);
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int64_t r = r1 + 32 * i, to = at + __popc(votes[i] & before);
            at += __popc(votes[i]);
            if (label[i] != a.ignore) {
                if (map) map[to] = static_cast<int>(r);
                if (!write) continue;
                w.map[to] = static_cast<int>(r);
                w.labels[to] = label[i] >= 0 && label[i] < a.vocab ? static_cast<int>(label[i]) : -1;
                if (backward) {
                    w.lse[to] = lse[i] * kL2E;
                    w.coef[to] = d[i] + e[i];
                    w.onehot[to] = d[i];
                    const float size = fabsf(d[i]) + fabsf(e[i]);
                    if (size < INFINITY) {  // (a row whose coefficients are no numbers has no say in the others' scale)
                        most = fmaxf(most, size);
                        most_d = fmaxf(most_d, fabsf(d[i]));
                    }
                }
            } else if (write && !backward && r < a.rows) {
                a.losses[r] = 0.0f;
                if (a.lse) a.lse[r] = 0.0f;
            }
        }
    }
    if (write) {
        most = warp_allreduce<MaxOp, 32>(most);
        most_d = warp_allreduce<MaxOp, 32>(most_d);
        if (lane == 0) warp_most[0][warp] = most, warp_most[1][warp] = most_d;
    }
    __syncthreads();
    if (write && warp == 0) {
        most = warp_allreduce<MaxOp, 32>(warp_most[0][lane]);
        most_d = warp_allreduce<MaxOp, 32>(warp_most[1][lane]);
        if (lane == 0) {
            // dz is divided by the largest coefficient and brought to 2^14 (at most 2^15 with that of the lse), where float16 has
            // room for small probabilities; and where all rows count alike, the label's -1 is a number that rounds to itself.
            float by = 1.0f, times = 1.0f;
            if (most > 0.0f) {
                const bool alike = most <= 2.0f * most_d;
                by = fminf(fmaxf(alike ? most_d : most, 0x1p-100f), 0x1p100f);
                times = alike ? 0x1p14f : 0x1p15f;
            }
            w.head->count = count;
            w.head->scale = times / by;
            w.head->unscale = a.logit_scale * (by / times);
        }
    }
    return count;
}
__global__ void __launch_bounds__(kScanThreads) rows_kernel(LossArgs a, Ws w, int backward) {
    pdl_release();
    pdl_enter();
    list_rows<8>(a, w, backward, true, nullptr);
}

// What is copied to rows of `pitch` elements that start on 16 bytes, 2 KB (of `chunks` in a row) by a warp at a time: rows that start
// elsewhere are read in the 16-byte words that cover them.
template <class T>
struct Packing {
    const T* src;
    T* dst;
    int64_t rows, pitch;
    int cols, chunks;
    // row `from` (below 0: zeros) to row r, its part `chunk`
    __device__ __forceinline__ void copy(int64_t r, int64_t from_row, int chunk) const {
        const int at = chunk * 128 + (threadIdx.x & 31), words = static_cast<int>(pitch / 8);
        uint4* to = reinterpret_cast<uint4*>(dst + r * pitch);
        uint4 q[4];
        if (from_row >= 0) {
            const uintptr_t p = reinterpret_cast<uintptr_t>(src + from_row * cols);
            const int shift = static_cast<int>(p & 15);
            const uint4* from = reinterpret_cast<const uint4*>(p - shift);
            const int have = (shift + 2 * cols + 15) / 16;  // words that cover the row
            if (shift == 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (at + 32 * j < have) q[j] = __ldg(from + at + 32 * j);
            } else {
                uint4 next[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = at + 32 * j;
                    q[j] = k < have ? __ldg(from + k) : make_uint4(0, 0, 0, 0);
                    next[j] = k + 1 < have ? __ldg(from + k + 1) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) q[j] = shifted(q[j], next[j], shift);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at + 32 * j < words) to[at + 32 * j] = q[j];
    }
};

// hidden's rows that have a loss, then zeros up to a whole block of the products' depth; all rows of the weight (its dst null: none);
// backward, the gradients of rows without a loss, which are zeros. SMALL: every CTA finds by itself which rows those are, and
// the first writes it down, so that one launch does all of it (up to 1024 rows).
template <class T, bool SMALL>
__global__ void __launch_bounds__(SMALL ? kScanThreads : kThreads) pack_kernel(LossArgs a, Ws w, int backward, Packing<T> hidden, Packing<T> weight) {
    __shared__ int small_map[SMALL ? kScanThreads : 1];
    pdl_release();
    pdl_enter();
    const int64_t count = SMALL ? list_rows<1>(a, w, backward, blockIdx.x == 0, small_map) : w.head->count;
    const int64_t end = (count + mma::kDepth - 1) / mma::kDepth * mma::kDepth * hidden.chunks;
    const int64_t all = end + (weight.dst ? weight.rows * weight.chunks : 0);
    const int64_t warps = blockDim.x / 32, step = gridDim.x * warps, first = blockIdx.x * warps + threadIdx.x / 32;
    for (int64_t i = first; i < all; i += step) {
        if (i < end) {
            const int64_t r = i / hidden.chunks;
            hidden.copy(r, r >= count ? -1 : SMALL ? small_map[r] : w.map[r], static_cast<int>(i - r * hidden.chunks));
        } else {
            const int64_t r = (i - end) / weight.chunks;
            weight.copy(r, r, static_cast<int>(i - end - r * weight.chunks));
        }
    }
    if (!backward || !a.dhidden) return;
    T* zeros = static_cast<T*>(a.dhidden);
    for (int64_t r = first; r < a.rows; r += step)
        if (a.labels[r] == a.ignore) zero_bytes(reinterpret_cast<char*>(zeros + r * a.cols), reinterpret_cast<char*>(zeros + (r + 1) * a.cols));
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
    mma::Boxes boxes;
    int cols, splits, width;
    int64_t first, n;
    float scale;      // log2(e) logit_scale
    int64_t rows;     // forward without packed rows
    const int64_t* labels;
    void* to;         // probs or dhidden
    void* dweight;
    int part;         // of the logits: see LossPlan
    int64_t pitch;    // of the rows of probs, of `sums`, or (forward) of the parts
    int second;       // where a row of probs has the second terms (0: nowhere)
    int fine_hidden, fine_weight;  // whether a gradient's products take them
    int begun, last;  // hidden gradient: whether the sums have earlier pieces, and whether this one completes them
    int wide, dweight_wide;  // rows of `to` and of dweight start on 16 bytes
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

// 32 columns of a row per lane, rounded to T, as half h of the rows of a box.
template <class T>
__device__ __forceinline__ void box_columns(const mma::OutBox& box, int h, const float (&v)[32]) {
#pragma unroll
    for (int g = 0; g < 4; ++g)
        box.put(4 * h + g, pack2<T>(v[8 * g], v[8 * g + 1]), pack2<T>(v[8 * g + 2], v[8 * g + 3]), pack2<T>(v[8 * g + 4], v[8 * g + 5]),
                pack2<T>(v[8 * g + 6], v[8 * g + 7]));
}

// 32 columns from c on of a row per lane that starts on 16 bytes (null: none), of which those below `cols` are written, rounded to T.
template <class T>
__device__ __forceinline__ void store_columns(T* row, int c, int cols, const float (&v)[32]) {
    if (!row) return;
#pragma unroll
    for (int g = 0; g < 4; ++g)
        if (c + 8 * g < cols)
            *reinterpret_cast<uint4*>(row + c + 8 * g) = make_uint4(pack2<T>(v[8 * g], v[8 * g + 1]), pack2<T>(v[8 * g + 2], v[8 * g + 3]),
                                                                    pack2<T>(v[8 * g + 4], v[8 * g + 5]), pack2<T>(v[8 * g + 6], v[8 * g + 7]));
}
// The same for rows that start anywhere: the columns are turned in the warp's room, so that it writes 32 of one row at a time; row(i), asked for
// in order, is where the warp's i-th row starts (null: none). (Words of four bytes, after an exchange between lanes where rows start between
// two, made the gradients of 64 x 2047 x 30000 225 us instead of 178.)
template <class T, class Row>
__device__ __forceinline__ void turn_columns(const mma::OutBox& box, Row&& row, int c, int cols, const float (&v)[32]) {
    const int lane = threadIdx.x & 31;
    box.clear();
    // (element i of row r lies at i ^ r of its row: no two lanes meet in a bank)
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("st.shared.f32 [%0], %1;" ::"r"(box.at + (lane * 32 + (i ^ lane)) * 4), "f"(v[i]) : "memory");
    __syncwarp();
    float f[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[i]) : "r"(box.at + (i * 32 + (lane ^ i)) * 4) : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        T* p = row(i);
        if (p && c + lane < cols) p[c + lane] = from_float<T>(f[i]);
    }
}

__device__ __forceinline__ void spoil(float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = NAN;
}

// Forward: (maximum, sum of 2^(z - maximum)) of each half of a tile's columns, and the label's z. The logits are summed in parts
// of p.part blocks of the depth, which are added in registers (see mma::run): a thread has 128 columns of a row.

// Two products, and two sums, in one instruction each.
__device__ __forceinline__ void pair_times(float& a, float& b, float by) {
    asm("{\n\t.reg .b64 v, w;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 w, {%2, %2};\n\tmul.rn.f32x2 v, v, w;\n\tmov.b64 {%0, %1}, v;\n\t}" : "+f"(a), "+f"(b) : "f"(by));
}
__device__ __forceinline__ void pair_plus(float& a, float& b, float c, float d) {
    asm("{\n\t.reg .b64 v, w;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 w, {%2, %3};\n\tadd.rn.f32x2 v, v, w;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d));
}

// A row's (maximum, sum) over a thread's columns below `limit` (WHOLE: all 128), z of which is the sum times scale; z of the column
// `label`, when that is one of them, is written to `picked`.
template <bool WHOLE>
__device__ __forceinline__ float2 max_and_sum(float (&z)[128], float scale, bool ok, int limit, int label, float* picked) {
    float m = -INFINITY;
#pragma unroll
    for (int c = 0; c < 128; c += 32) {
        if (!WHOLE && c >= limit) continue;
#pragma unroll
        for (int i = c; i < c + 32; i += 2) {
            pair_times(z[i], z[i + 1], scale);
            if (!WHOLE && i >= limit) z[i] = -INFINITY;
            if (!WHOLE && i + 1 >= limit) z[i + 1] = -INFINITY;
            m = fmaxf(m, fmaxf(z[i], z[i + 1]));
        }
        if (label >= c && label < c + 32) {
#pragma unroll
            for (int i = c; i < c + 32; ++i)
                if (label == i) *picked = z[i];
        }
    }
    const float from = m == -INFINITY ? 0.0f : m;
    float s[8] = {};
#pragma unroll
    for (int c = 0; c < 128; c += 32) {
        if (!WHOLE && c >= limit) continue;
#pragma unroll
        for (int g = c; g < c + 32; g += 8) {
            float part[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = g; i < g + 8; i += 2) {
                pair_plus(z[i], z[i + 1], -from, -from);
                z[i] = ex2(z[i]);
                z[i + 1] = ex2(z[i + 1]);
                pair_plus(part[0], part[1], z[i], z[i + 1]);
            }
            pair_plus(s[g / 4 & 6], s[(g / 4 & 6) + 1], part[0], part[1]);
        }
    }
    return make_float2(ok ? m : NAN, ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])));
}

template <class T>
__global__ void __cluster_dims__(2) __launch_bounds__(mma::kThreads, 1)
    stats_kernel(const __grid_constant__ CUtensorMap hidden, const __grid_constant__ CUtensorMap weight, const __grid_constant__ Product p) {
    int64_t count = 0;
    float z[128];
    const mma::Operands<false, false> o{&hidden, &weight};
    mma::run<mma::kEach>(
        o, o, p.boxes, kTypeBits<T>, p.lim, p.part,
        [&] {
            count = p.w.map ? p.w.head->count : p.rows;
            return mma::Work(p.width, mma::Tiles{tiles_of(count, kTileRows), tiles_of(p.n, p.width), 1, tiles_of(p.cols, mma::kDepth)});
        },
        [&](const mma::Unit& u, int row, int half, int first, int last, uint32_t at, bool ok, const mma::OutBox&, bool begun, bool whole, auto&& release) {
            if (row - static_cast<int>(threadIdx.x & 31) >= count) return release();  // none of the warp's rows is one
            const int limit = static_cast<int>(min(static_cast<int64_t>(last), p.n - u.n)) - first;  // columns of the vocabulary
            int label = -1;  // (asked for early: it is on its way while the columns come)
            if (whole && row < count) {
                if (p.w.map) {
                    label = p.w.labels[row];
                } else {
                    const int64_t l = p.labels[row];
                    label = l >= 0 && l < p.n ? static_cast<int>(l) : -1;
                }
            }
            mma::take_part(at + first, limit, begun, z);
            release();
            if (!whole) return;
            label = label >= u.n + first && label < u.n + first + limit ? label - u.n - first : -1;
            const float2 part = limit >= 128 ? max_and_sum<true>(z, p.scale, ok, limit, label, p.w.picked + row)
                                             : max_and_sum<false>(z, p.scale, ok, limit, label, p.w.picked + row);
            if (row < count) p.w.parts[row * p.pitch + 2 * (u.n / p.width) + half] = part;
        });
}

// Backward: scale dz / logit_scale of a piece, rounded, and (FINE) what the rounding left. The logits are summed in the forward pass's parts, so that they
// are the very numbers that the lse was formed from: a row whose label has all of the probability has a dz of 0, not of the error of a sum.
// Rows and words beyond the last are zeros up to the tile's end.
template <class T, bool FINE>
__global__ void __cluster_dims__(2) __launch_bounds__(mma::kThreads, 1)
    probs_kernel(const __grid_constant__ CUtensorMap hidden, const __grid_constant__ CUtensorMap weight, const __grid_constant__ CUtensorMap out,
                 const __grid_constant__ Product p) {
    int64_t count = 0;
    float times = 0.0f, z[128];
    const mma::Operands<false, false> o{&hidden, &weight};
    mma::run<mma::kEach>(
        o, o, p.boxes, kTypeBits<T>, p.lim, p.part,
        [&] {
            count = p.w.head->count;
            times = p.w.head->scale;
            return mma::Work(p.width, mma::Tiles{tiles_of(count, kTileRows), tiles_of(p.n, p.width), 1, tiles_of(p.cols, mma::kDepth)});
        },
        [&](const mma::Unit& u, int row, int, int first, int last, uint32_t at, bool ok, const mma::OutBox& box, bool begun, bool whole, auto&& release) {
            // rows that are not there are read as the depth of the weight's gradient up to the end of a block
            const int row0 = row - static_cast<int>(threadIdx.x & 31);
            if (row0 >= (count + mma::kDepth - 1) / mma::kDepth * mma::kDepth) return release();
            const bool in = row < count;
            const int limit = static_cast<int>(min(static_cast<int64_t>(last), p.n - u.n)) - first;
            float lse = 0.0f, coef = 0.0f, onehot = 0.0f;
            int word = -1;
            if (whole && in) {  // (asked for early, as above)
                lse = p.w.lse[row];
                coef = p.w.coef[row] * times;
                onehot = p.w.onehot[row] * times;
                word = p.w.labels[row];
            }
            mma::take_part(at + first, last - first, begun, z);
            release();
            if (!whole) return;
            const int label = word >= 0 ? static_cast<int>(word - p.first) - u.n - first : -1;
            const bool boxed = (last - first) % 64 == 0;
            const auto store = [&](const float(&v)[32], int c, int term) {
                if (boxed) {
                    const int h = c / 32 & 1;
                    if (h == 0) box.clear();
                    box_columns<T>(box, h, v);
                    if (h == 1) box.send(&out, term + u.n + first + c - 32, row0);
                } else {
                    store_columns<T>(static_cast<T*>(p.to) + row * p.pitch + term + u.n + first, c, last - first, v);
                }
            };
#pragma unroll
            for (int c = 0; c < 128; c += 32) {
                if (c >= last - first) continue;
                float(&v)[32] = *reinterpret_cast<float(*)[32]>(z + c);
                if (!ok) spoil(v);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = coef * ex2(fmaf(v[i], p.scale, -lse));
                if (label >= c && label < c + 32) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (label == c + i) v[i] -= onehot;
                }
                if (!in || c + 32 > limit) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!in || c + i >= limit) v[i] = 0.0f;
                }
                store(v, c, 0);
            }
            if constexpr (!FINE) return;
#pragma unroll
            for (int c = 0; c < 128; c += 32) {  // what the rounding left, which is exact before its own
                if (c >= last - first) continue;
                float(&v)[32] = *reinterpret_cast<float(*)[32]>(z + c);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] -= to_float(from_float<T>(v[i]));
                store(v, c, p.second);
            }
        });
}

// Backward: the piece's part of the hidden gradient, added to those of earlier pieces (the last one writes the gradient), and
// the piece's rows of the weight's gradient. One launch has both, so that there is one end at which pairs run out of work.
template <class T>
__device__ __forceinline__ void hidden_part(const Product& p, const mma::Unit& u, int64_t count, float times, int row, int first, int last, uint32_t at,
                                            bool ok, const mma::OutBox& box) {
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
            const int n = min(last, p.cols - u.n);
            if (p.wide) store_columns<T>(to, c, n, z);
            else
                turn_columns<T>(
                    box, [&](int i) { return reinterpret_cast<T*>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(to), i)); }, c, n, z);
        }
    }
}
template <class T>
__device__ __forceinline__ void weight_part(const Product& p, const CUtensorMap* out, const mma::Unit& u, float times, int row, int first, int last,
                                            uint32_t at, bool ok, const mma::OutBox& box) {
    const int row0 = row - static_cast<int>(threadIdx.x & 31), cols = min(last, p.cols - u.n);
    T* to = static_cast<T*>(p.dweight) + (p.first + row0) * p.cols + u.n;
    const int have = static_cast<int>(min(int64_t{32}, p.n - row0));
    for (int c = first; c < cols; c += 32) {
        float z[32];
        mma::load_columns(at + c, z);
        if (!ok) spoil(z);
#pragma unroll
        for (int i = 0; i < 32; ++i) z[i] = u.begin == u.end ? 0.0f : z[i] * times;
        if (p.dweight_wide) {  // (what a box has beyond the last row and column is not written)
            const int h = (c - first) / 32 & 1;
            if (h == 0) box.clear();
            box_columns<T>(box, h, z);
            if (h == 1 || c + 32 >= cols) box.send(out, u.n + c - 32 * h, row0);
        } else {
            turn_columns<T>(
                box,
                [&p, have, q = to](int i) mutable {
                    T* at = i < have ? q : nullptr;
                    q += p.cols;
                    return at;
                },
                c, cols, z);
        }
    }
}
template <class T, bool LONG>
__global__ void __cluster_dims__(2) __launch_bounds__(mma::kThreads, 1)
    grads_kernel(const __grid_constant__ CUtensorMap probs_rows, const __grid_constant__ CUtensorMap weight, const __grid_constant__ CUtensorMap probs_cols,
                 const __grid_constant__ CUtensorMap hidden, const __grid_constant__ CUtensorMap dweight_out, const __grid_constant__ Product p) {
    int64_t count = 0;
    float times = 0.0f;
    mma::Operands<false, true> of_hidden{&probs_rows, &weight};
    mma::Operands<true, true> of_weight{&probs_cols, &hidden};
    of_hidden.second = of_weight.second = p.second;
    mma::run<LONG ? mma::kJoined : mma::kWhole>(
        of_hidden, of_weight, p.boxes, kTypeBits<T>, p.lim, kGradPart,
        [&] {
            count = p.w.head->count;
            times = p.w.head->unscale;
            const int across = tiles_of(p.cols, p.width);
            mma::Tiles dhidden, dweight;
            of_hidden.blocks = tiles_of(p.n, mma::kDepth);
            of_weight.blocks = tiles_of(count, mma::kDepth);
            if (p.to) dhidden = mma::Tiles{tiles_of(count, kTileRows), across, p.splits, of_hidden.blocks << p.fine_hidden};
            if (p.dweight) dweight = mma::Tiles{tiles_of(p.n, kTileRows), across, 1, of_weight.blocks << p.fine_weight};
            return mma::Work(p.width, dhidden, dweight);
        },
        [&](const mma::Unit& u, int row, int, int first, int last, uint32_t at, bool ok, const mma::OutBox& box, bool, bool, auto&& release) {
            const int row0 = row - static_cast<int>(threadIdx.x & 31);
            if (u.kind == 1) {
                if (row0 < p.n) weight_part<T>(p, &dweight_out, u, times, row, first, last, at, ok, box);
            } else if (row0 < count) {
                hidden_part<T>(p, u, count, times, row, first, last, at, ok, box);
            }
            release();
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

// The parts of a row's sum joined by a warp: the maximum first, then the sums about it.
__global__ void __launch_bounds__(kThreads) join_kernel(LossArgs a, Ws w, int parts) {
    pdl_enter();
    const int64_t count = w.map ? w.head->count : a.rows;
    const int lane = threadIdx.x & 31, warps = kThreads / 32;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * warps + (threadIdx.x >> 5); r < count; r += static_cast<int64_t>(gridDim.x) * warps) {
        const float2* part = w.parts + r * parts;
        const int64_t to = w.map ? w.map[r] : r, given = w.map ? w.labels[r] : a.labels[r];
        const bool labelled = given >= 0 && given < a.vocab, gone = !w.map && given == a.ignore;
        const float picked = labelled ? w.picked[r] : 0.0f;
        float m = -INFINITY, s = 0.0f;
        for (int i0 = 0; i0 < parts; i0 += 32 * 16) {
            float2 p[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int i = i0 + 32 * j + lane;
                p[j] = i < parts ? part[i] : make_float2(-INFINITY, 0.0f);
            }
            float most = m;
#pragma unroll
            for (int j = 0; j < 16; ++j) most = fmaxf(most, p[j].x);
            const float from = most == -INFINITY ? 0.0f : most;
            s *= ex2(m - from);
#pragma unroll
            for (int j = 0; j < 16; ++j) s = fmaf(p[j].y, ex2(p[j].x - from), s);
            m = most;
        }
        const float most = warp_allreduce<MaxOp, 32>(m);
        s = warp_allreduce<SumOp, 32>(s * ex2(m - (most == -INFINITY ? 0.0f : most)));
        if (lane == 0) {
            const float log = logf(s), lse = fmaf(most, kLN2, log);
            a.losses[to] = gone ? 0.0f : labelled ? fmaf(most - picked, kLN2, log) : lse;
            if (a.lse) a.lse[to] = gone ? 0.0f : lse;
        }
    }
}

Ws workspace(const LossArgs& a, const LossPlan& p) {
    auto f = [&](size_t at) { return reinterpret_cast<float*>(a.ws + at); };
    return Ws{reinterpret_cast<LossHead*>(a.ws + p.head), reinterpret_cast<int*>(a.ws + p.map), reinterpret_cast<int*>(a.ws + p.labels),
              f(p.lse), f(p.coef), f(p.onehot), reinterpret_cast<float2*>(a.ws + p.parts_at), f(p.picked), f(p.sums), p.rows_pad};
}

// hidden's rows that have a loss, and the weight where its rows do not start on 16 bytes.
template <class T>
cudaError_t pack(const LossArgs& a, const LossPlan& p, const Ws& w, int backward, const T** hidden, const T** weight, cudaStream_t stream) {
    const int chunks = static_cast<int>(ceil_div(p.pitch, 1024));
    Packing<T> h{static_cast<const T*>(a.hidden), reinterpret_cast<T*>(a.ws + p.hidden), a.rows, p.pitch, a.cols, chunks};
    Packing<T> t{static_cast<const T*>(a.weight), p.pack_weight ? reinterpret_cast<T*>(a.ws + p.weight) : nullptr, a.vocab, p.pitch, a.cols, chunks};
    *hidden = h.dst;
    *weight = t.dst ? t.dst : t.src;
    const int64_t items = (a.rows + mma::kDepth + (t.dst ? a.vocab : 0)) * chunks;
    if (a.rows <= kScanThreads) {
        const int64_t ctas = std::min<int64_t>(ceil_div(items, kScanThreads / 32), 4 * kPairs);
        return launch_dependent(pack_kernel<T, true>, dim3(static_cast<unsigned>(ctas)), kScanThreads, 0, 1, stream, a, w, backward, h, t);
    }
    const cudaError_t e = launch_dependent(rows_kernel, dim3(1), kScanThreads, 0, 1, stream, a, w, backward);
    if (e != cudaSuccess) return e;
    const int64_t ctas = std::min<int64_t>(ceil_div(items, kThreads / 32), 1 << 14);
    return launch_dependent(pack_kernel<T, false>, dim3(static_cast<unsigned>(ctas)), kThreads, 0, 1, stream, a, w, backward, h, t);
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
template <class K, class... A>
cudaError_t launch_product(K kernel, int64_t units, cudaStream_t stream, const A&... args) {
    const int resident = resident_ctas(reinterpret_cast<const void*>(kernel), mma::kThreads, mma::kSmem, 2);
    if (resident < 2) return cudaErrorInvalidConfiguration;
    const int64_t pairs = std::min<int64_t>(units, resident / 2);
    return launch_dependent(kernel, dim3(static_cast<unsigned>(2 * pairs)), mma::kThreads, mma::kSmem, 1, stream, args...);
}

template <class T>
cudaError_t forward(const LossArgs& a, cudaStream_t stream) {
    const LossPlan p(a.rows, a.cols, a.vocab, false);
    Ws w = workspace(a, p);
    // One tile of rows is not shorter without the rows that have no loss: they are read where they are.
    const bool direct = a.rows <= kTileRows && a.cols % 8 == 0 && reinterpret_cast<uintptr_t>(a.hidden) % 16 == 0;
    const T *from = static_cast<const T*>(a.hidden), *table = static_cast<const T*>(a.weight);
    cudaError_t e = cudaSuccess;
    if (direct) w.map = nullptr;
    else e = pack<T>(a, p, w, 0, &from, &table, stream);
    const mma::Boxes boxes = mma::boxes_for(a.rows);
    CUtensorMap hidden, weight;
    if (e == cudaSuccess) e = map_of(&hidden, from, direct ? a.rows : p.rows_pad, a.cols, p.pitch, boxes.rows);
    if (e == cudaSuccess) e = map_of(&weight, table, a.vocab, a.cols, p.pitch, p.width / 2);
    if (e != cudaSuccess) return e;
    Product d{};
    d.w = w;
    d.lim = mma::Limits{device_error_word(), debug_flags_now()};
    d.boxes = boxes;
    d.cols = a.cols;
    d.width = p.width;
    d.n = a.vocab;
    d.scale = a.logit_scale * kL2E;
    d.rows = a.rows;
    d.labels = a.labels;
    d.part = p.logit_part;
    d.pitch = p.parts;
    e = launch_product(stats_kernel<T>, p.rows_pad / kTileRows * ceil_div(a.vocab, p.width), stream, hidden, weight, d);
    if (e != cudaSuccess) return e;
    const int64_t ctas = std::min<int64_t>(ceil_div(a.rows, kThreads / 32), 1 << 16);
    return launch_dependent(join_kernel, dim3(static_cast<unsigned>(ctas)), kThreads, 0, 1, stream, a, w, static_cast<int>(p.parts));
}

template <class T>
cudaError_t backward(const LossArgs& a, cudaStream_t stream) {
    const LossPlan p(a.rows, a.cols, a.vocab, true);
    const Ws w = workspace(a, p);
    const T *hidden, *weight;
    cudaError_t e = pack<T>(a, p, w, 1, &hidden, &weight, stream);
    T* probs = reinterpret_cast<T*>(a.ws + p.probs);
    const mma::Boxes boxes = mma::boxes_for(a.rows);
    CUtensorMap hidden_rows, hidden_cols, probs_rows, probs_cols, probs_out;
    if (e == cudaSuccess) e = map_of(&hidden_rows, hidden, p.rows_pad, a.cols, p.pitch, boxes.rows);
    if (e == cudaSuccess) e = map_of(&hidden_cols, hidden, p.rows_pad, a.cols, p.pitch, mma::kDepth);
    const int64_t dz_pitch = p.piece * p.terms;
    if (e == cudaSuccess) e = map_of(&probs_rows, probs, p.rows_pad, dz_pitch, dz_pitch, boxes.rows);
    if (e == cudaSuccess) e = map_of(&probs_cols, probs, p.rows_pad, dz_pitch, dz_pitch, mma::kDepth);
    if (e == cudaSuccess) e = map_of(&probs_out, probs, p.rows_pad, dz_pitch, dz_pitch, 32);
    const int64_t row_tiles = p.rows_pad / kTileRows;
    const bool align = a.cols % 8 == 0, dweight_wide = a.dweight && align && reinterpret_cast<uintptr_t>(a.dweight) % 16 == 0;
    for (int64_t first = 0; first < a.vocab && e == cudaSuccess; first += p.piece) {
        const int64_t n = std::min(p.piece, a.vocab - first);
        CUtensorMap weight_rows, weight_cols, dweight_out = probs_out;
        e = map_of(&weight_rows, weight + first * p.pitch, n, a.cols, p.pitch, p.width / 2);
        if (e == cudaSuccess) e = map_of(&weight_cols, weight + first * p.pitch, n, a.cols, p.pitch, mma::kDepth);
        if (e == cudaSuccess && dweight_wide) e = map_of(&dweight_out, static_cast<const T*>(a.dweight) + first * a.cols, n, a.cols, a.cols, 32);
        if (e != cudaSuccess) break;
        Product d{};
        d.w = w;
        d.lim = mma::Limits{device_error_word(), debug_flags_now()};
        d.boxes = boxes;
        d.cols = a.cols;
        d.first = first;
        d.n = n;
        d.scale = a.logit_scale * kL2E;
        d.width = p.width;
        d.to = probs;
        d.pitch = dz_pitch;
        d.part = p.logit_part;
        d.second = p.terms > 1 ? static_cast<int>(p.piece) : 0;
        d.fine_hidden = p.fine_hidden;
        d.fine_weight = p.fine_weight;
        const auto probs_of = p.terms > 1 ? probs_kernel<T, true> : probs_kernel<T, false>;
        e = launch_product(probs_of, row_tiles * ceil_div(n, p.width), stream, hidden_rows, weight_rows, probs_out, d);
        if (e != cudaSuccess) break;
        const int64_t across = ceil_div(a.cols, p.grad_width);
        d.width = p.grad_width;
        d.splits = p.splits;
        d.to = a.dhidden;
        d.dweight = a.dweight;
        d.pitch = p.pitch;
        d.begun = first > 0;
        d.last = p.splits == 1 && first + n == a.vocab;
        d.wide = align && reinterpret_cast<uintptr_t>(a.dhidden) % 16 == 0;
        d.dweight_wide = dweight_wide;
        const int64_t units = (a.dhidden ? row_tiles * across * p.splits : 0) + (a.dweight ? ceil_div(n, kTileRows) * across : 0);
        const auto grads_of = p.parted ? grads_kernel<T, true> : grads_kernel<T, false>;
        e = launch_product(grads_of, units, stream, probs_rows, weight_cols, probs_cols, hidden_cols, dweight_out, d);
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
