// Embedding lookup and its gradient by sorted tokens.
//
// Forward: out[t] = scale table[ids[t]]. Lanes take 16 bytes, four loads under way together. Bound by memory: 16384 x 4096 bf16 32 us
// (frequent rows come from L2), 6039 x 1537 float32 10 us.
//
// Backward: dtable[v] = scale (the sum of dy[t] over the tokens t with ids[t] = v). The tokens are sorted
// by id with a stable radix sort, so that a row's terms come in the order of the tokens and the sums
// repeat bit for bit without atomics. Then a warp sums the rows whose segment starts
// in its 32 sorted tokens, 512 bytes of columns wide, in binary32. Segments longer than 64 tokens
// are cut at the tiles' borders into partial sums, which a last kernel adds in order, so one frequent token
// costs no more than many rare ones. The zeros of rows that no token has are written beside both: as many as
// fit beside the sort of one CTA, the others beside the sums. Bound by memory, most of it the zeros: 16384 x 4096 bf16 into 50257 rows
// 105 us (the bytes that cannot be avoided take 82 at the copy rate; zeros alone are written at 6.0 of its 6.7 TB/s),
// 6039 x 1537 f16 into float32 72 us (49). Added to a table, where no zeros hide the sort: 16384 x 4096 bf16 109 us; into 5003 rows 77, added 94. More than
// 16384 tokens are sorted by several CTAs in three launches for each eight bits of the ids, 34 us for 131072.
#include <algorithm>

#include "tr_launch.h"
#include "tr_vocab.cuh"
#include "tr_vocab.h"

namespace tr {
namespace vocab {

using block::from_float;
using block::to_float;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// N elements of T as one access of a lane: 16 bytes of the narrowest type, or one element.
template <class T, int N>
__device__ __forceinline__ void load_floats(const T* p, float (&v)[N]) {
    if constexpr (N == 1) {
        v[0] = to_float(*p);
    } else {
        static_assert(N * sizeof(T) % 16 == 0, "whole 16-byte words");
#pragma unroll
        for (int j = 0; j < N * static_cast<int>(sizeof(T)) / 16; ++j) {
            const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + j);
            constexpr int kPer = 16 / sizeof(T);
            T e[kPer];
            memcpy(e, &q, 16);
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[j * kPer + i] = to_float(e[i]);
        }
    }
}
template <class T, int N>
__device__ __forceinline__ void store_floats(T* p, const float (&v)[N]) {
    if constexpr (N == 1) {
        *p = from_float<T>(v[0]);
    } else {
#pragma unroll
        for (int j = 0; j < N * static_cast<int>(sizeof(T)) / 16; ++j) {
            constexpr int kPer = 16 / sizeof(T);
            T e[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) e[i] = from_float<T>(v[j * kPer + i]);
            uint4 q;
            memcpy(&q, e, 16);
            reinterpret_cast<uint4*>(p)[j] = q;
        }
    }
}

// ---- forward ---------------------------------------------------------------------

template <class T>
constexpr int kLane = 16 / sizeof(T);  // elements of 16 bytes

// 16 bytes of a row times scale.
template <class T>
__device__ __forceinline__ uint4 scaled(const uint4& q, float scale) {
    T e[kLane<T>];
    memcpy(e, &q, 16);
#pragma unroll
    for (int i = 0; i < kLane<T>; ++i) e[i] = from_float<T>(scale * to_float(e[i]));
    uint4 r;
    memcpy(&r, e, 16);
    return r;
}

// Rows of at least 1 KB that start on 16 bytes: a warp takes 2 KB of one.
template <class T>
__global__ void __launch_bounds__(kThreads) embed_kernel(EmbedArgs a, int chunks) {
    pdl_enter();
    const int lane = threadIdx.x & 31, words = a.cols / kLane<T>;
    const int64_t items = a.tokens * chunks;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < items;
         i += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t token = i / chunks;
        const int first = static_cast<int>(i - token * chunks) * 128 + lane;
        const int64_t id = __ldg(a.ids + token);
        const bool inside = id >= 0 && id < a.vocab;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(a.table) + (inside ? id : 0) * a.cols);
        uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + token * a.cols);
        uint4 q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = inside && first + 32 * j < words ? __ldg(src + first + 32 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (first + 32 * j < words) dst[first + 32 * j] = inside ? scaled<T>(q[j], a.scale) : q[j];
    }
}

// Shorter ones: a thread takes 16 bytes of four rows (131072 x 128 bf16: 8 us, by the kernel above 33).
template <class T>
__global__ void __launch_bounds__(kThreads) embed_short_kernel(EmbedArgs a) {
    pdl_enter();
    const uint32_t words = a.cols / kLane<T>;
    const int64_t items = a.tokens * words;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * (4 * kThreads) + threadIdx.x; i0 < items; i0 += static_cast<int64_t>(gridDim.x) * (4 * kThreads)) {
        int64_t id[4];
        uint32_t word[4];
        uint4 q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t i = i0 + j * kThreads, token = i >> 32 ? i / words : static_cast<uint32_t>(i) / words;
            word[j] = static_cast<uint32_t>(i - token * words);
            id[j] = i < items ? __ldg(a.ids + token) : -1;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            q[j] = make_uint4(0, 0, 0, 0);
            if (id[j] >= 0 && id[j] < a.vocab) q[j] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.table) + id[j] * a.cols) + word[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool inside = id[j] >= 0 && id[j] < a.vocab;
            if (i0 + j * kThreads < items) reinterpret_cast<uint4*>(a.out)[i0 + j * kThreads] = inside ? scaled<T>(q[j], a.scale) : q[j];
        }
    }
}

// float32 rows that start anywhere: a warp takes 256 elements, 32 apart for a lane (8192 x 4095: 33 us, by the kernel below 35).
__global__ void __launch_bounds__(kThreads) embed_floats_kernel(EmbedArgs a, int chunks) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t items = a.tokens * chunks;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < items;
         i += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t token = i / chunks;
        const int first = static_cast<int>(i - token * chunks) * 256 + lane;
        const int64_t id = __ldg(a.ids + token);
        const bool inside = id >= 0 && id < a.vocab;
        const float* src = static_cast<const float*>(a.table) + (inside ? id : 0) * a.cols;
        float* dst = static_cast<float*>(a.out) + token * a.cols;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = inside && first + 32 * j < a.cols ? __ldg(src + first + 32 * j) : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (first + 32 * j < a.cols) dst[first + 32 * j] = inside ? a.scale * v[j] : 0.0f;
    }
}

// 16-bit rows that start anywhere: the 16-byte words of the output row, each from the two words of the table that cover it, and the elements
// before the first and after the last.
template <class T>
__global__ void __launch_bounds__(kThreads) embed_odd_kernel(EmbedArgs a, int chunks) {
    pdl_enter();
    constexpr int kSize = sizeof(T);
    const int lane = threadIdx.x & 31;
    const int64_t items = a.tokens * chunks;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < items;
         i += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t token = i / chunks;
        const int chunk = static_cast<int>(i - token * chunks);
        const int64_t id = __ldg(a.ids + token);
        const bool inside = id >= 0 && id < a.vocab;
        const T* src = static_cast<const T*>(a.table) + (inside ? id : 0) * a.cols;
        T* dst = static_cast<T*>(a.out) + token * a.cols;
        const int head = min(a.cols, static_cast<int>(-reinterpret_cast<uintptr_t>(dst) & 15) / kSize), words = (a.cols - head) / kLane<T>;
        const uintptr_t body = reinterpret_cast<uintptr_t>(src + head);
        const int shift = static_cast<int>(body & 15);
        const uint4* from = reinterpret_cast<const uint4*>(body - shift);
        uint4* to = reinterpret_cast<uint4*>(dst + head);
        uint4 lo[4], hi[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = chunk * 128 + lane + 32 * j;
            const bool in = inside && k < words;
            lo[j] = in ? __ldg(from + k) : make_uint4(0, 0, 0, 0);
            hi[j] = in && shift ? __ldg(from + k + 1) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = chunk * 128 + lane + 32 * j;
            if (k < words) to[k] = inside ? scaled<T>(shifted(lo[j], hi[j], shift), a.scale) : lo[j];
        }
        if (chunk == 0) {  // the ends, fewer than 16 elements
            const int end = head + words * kLane<T>, n = head + a.cols - end;
            if (lane < n) {
                const int c = lane < head ? lane : end + lane - head;
                dst[c] = from_float<T>(inside ? a.scale * to_float(src[c]) : 0.0f);
            }
        }
    }
}

// ---- the sort ----------------------------------------------------------------------

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortItems = kSortTile / kSortThreads;  // of a thread, at most
constexpr uint32_t kNoKey = 0xffffffffu;  // beyond every id: the places after the last token

// Shared memory of a sorting CTA: of a pass, and of a whole sort.
struct PassShared {
    uint32_t hist[kSortWarps][kSortBins];
    uint32_t base[kSortBins];
};
struct SortShared : PassShared {
    uint32_t key[kSortTile];
    uint16_t place[kSortTile];
};

// A token's key: its id, or `vocab` (behind every id) when that is outside the table.
__device__ __forceinline__ uint32_t key_of(const EmbedGradArgs& a, int64_t t) {
    const int64_t id = __ldg(a.ids + t);
    return static_cast<uint32_t>(id >= 0 && id < a.vocab ? id : a.vocab);
}

// Item i of a thread's ITEMS: a warp's items are consecutive.
template <int ITEMS>
__device__ __forceinline__ int item_of(int i) {
    return (threadIdx.x >> 5) * (32 * ITEMS) + i * 32 + (threadIdx.x & 31);
}

// rank[i] = how many items of the tile that come before item i have its digit, once base is added:
// s.hist[w][d] becomes the count of digit d in the warps before w, and `count` (thread d < 256) the tile's
// count of digit d. Begins and ends with a barrier.
template <int ITEMS>
__device__ __forceinline__ uint32_t rank_digits(const uint32_t (&key)[ITEMS], int shift, uint32_t (&rank)[ITEMS], PassShared& s) {
    const int warp = threadIdx.x >> 5;
    const unsigned before = (1u << (threadIdx.x & 31)) - 1u;
    __syncthreads();
    for (int b = threadIdx.x; b < kSortWarps * kSortBins; b += kSortThreads) (&s.hist[0][0])[b] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const uint32_t d = (key[i] >> shift) & (kSortBins - 1);
        unsigned same = kFull;  // the lanes with this digit (votes on its bits: 37 us for 16384 tokens, with __match_any_sync 39)
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const unsigned vote = __ballot_sync(kFull, d >> b & 1);
            same &= d >> b & 1 ? vote : ~vote;
        }
        const uint32_t old = s.hist[warp][d];
        __syncwarp();
        if ((same & before) == 0) s.hist[warp][d] = old + __popc(same);
        __syncwarp();
        rank[i] = old + __popc(same & before);
    }
    __syncthreads();
    uint32_t count = 0;
    if (threadIdx.x < kSortBins) {
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t n = s.hist[w][threadIdx.x];
            s.hist[w][threadIdx.x] = count;
            count += n;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) rank[i] += s.hist[warp][(key[i] >> shift) & (kSortBins - 1)];
    return count;
}

// Exclusive sums over the threads below 256 (the other warps take part in the barriers).
__device__ __forceinline__ uint32_t bins_before(uint32_t n, uint32_t* warp_total) {
    uint32_t inc = n;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += v;
    }
    __syncthreads();
    if (warp < kSortBins / 32 && lane == 31) warp_total[warp] = inc;
    __syncthreads();
    uint32_t sum = inc - n;
#pragma unroll
    for (int w = 0; w < kSortBins / 32; ++w) sum += w < warp ? warp_total[w] : 0;
    return sum;
}

// Up to 1024 ITEMS tokens sorted by one CTA.
template <int ITEMS>
__device__ __forceinline__ void sort_one_tile(const EmbedGradArgs& a, int bits, uint32_t* keys, uint32_t* places,
                                              SortShared& s) {
    __shared__ uint32_t warp_total[kSortBins / 32];
    const int n = static_cast<int>(a.tokens);
    uint32_t key[ITEMS], rank[ITEMS];
    uint16_t place[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int t = item_of<ITEMS>(i);
        key[i] = t < n ? key_of(a, t) : kNoKey;
        place[i] = static_cast<uint16_t>(t);
    }
    for (int shift = 0; shift < bits; shift += 8) {
        const uint32_t count = rank_digits(key, shift, rank, s);
        const uint32_t base = bins_before(count, warp_total);
        if (threadIdx.x < kSortBins) s.base[threadIdx.x] = base;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const uint32_t at = s.base[(key[i] >> shift) & (kSortBins - 1)] + rank[i];
            s.key[at] = key[i];
            s.place[at] = place[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            key[i] = s.key[item_of<ITEMS>(i)];
            place[i] = s.place[item_of<ITEMS>(i)];
        }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int t = item_of<ITEMS>(i);
        if (t < n) {
            keys[t] = key[i];
            places[t] = place[i];
        }
    }
}

// One pass of a sort over several CTAs: the tiles' counts of each digit, their places, the scatter.
constexpr int kPassItems = kPassTile / kSortThreads;
struct SortPass {
    const uint32_t* keys;  // null: the first pass, from the ids
    const uint32_t* places;
    uint32_t* out_keys;
    uint32_t* out_places;
    uint32_t* counts;  // [bin][tile]
    uint32_t* listed;  // emptied
    int64_t tiles;
    int shift;
};

template <bool SCATTER>
__global__ void __launch_bounds__(kSortThreads) sort_pass_kernel(EmbedGradArgs a, SortPass p) {
    __shared__ PassShared s;
    pdl_enter();
    const int64_t tile = blockIdx.x;
    if (tile == 0 && threadIdx.x == 0) *p.listed = 0;
    uint32_t key[kPassItems], rank[kPassItems], place[kPassItems];
#pragma unroll
    for (int i = 0; i < kPassItems; ++i) {
        const int64_t t = tile * kPassTile + item_of<kPassItems>(i);
        key[i] = t < a.tokens ? (p.keys ? p.keys[t] : key_of(a, t)) : kNoKey;
        if (SCATTER) place[i] = t < a.tokens && p.places ? p.places[t] : static_cast<uint32_t>(t);
    }
    const uint32_t base = SCATTER && threadIdx.x < kSortBins ? p.counts[threadIdx.x * p.tiles + tile] : 0;
    const uint32_t count = rank_digits(key, p.shift, rank, s);
    if constexpr (!SCATTER) {
        if (threadIdx.x < kSortBins) p.counts[threadIdx.x * p.tiles + tile] = count;
    } else {
        if (threadIdx.x < kSortBins) s.base[threadIdx.x] = base;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPassItems; ++i) {
            if (tile * kPassTile + item_of<kPassItems>(i) >= a.tokens) continue;
            const uint32_t at = s.base[(key[i] >> p.shift) & (kSortBins - 1)] + rank[i];
            p.out_keys[at] = key[i];
            p.out_places[at] = place[i];
        }
    }
}

// Where each tile's items of each digit go: the counts' exclusive sums in order of digit and tile. (The last
// tile's missing items have digit 255 and are counted last, so they move nothing.)
__global__ void __launch_bounds__(kSortThreads) sort_scan_kernel(uint32_t* counts, int64_t tiles) {
    constexpr int kEach = 8;  // counts of a thread at a time
    __shared__ uint32_t warp_total[kSortWarps], carry_in;
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n = tiles * kSortBins;  // a multiple of kEach
    uint32_t carry = 0;
    for (int64_t at = 0; at < n; at += kEach * kSortThreads) {
        const int64_t i = at + kEach * static_cast<int64_t>(threadIdx.x);
        uint4 q[2] = {};
        if (i < n) q[0] = reinterpret_cast<const uint4*>(counts + i)[0], q[1] = reinterpret_cast<const uint4*>(counts + i)[1];
        uint32_t v[kEach], sum = 0;
        memcpy(v, q, sizeof(v));
#pragma unroll
        for (int j = 0; j < kEach; ++j) sum += v[j];
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += u;
        }
        if (lane == 31) warp_total[warp] = inc;
        __syncthreads();
        uint32_t before = carry + inc - sum;
        for (int w = 0; w < warp; ++w) before += warp_total[w];
        if (threadIdx.x == kSortThreads - 1) carry_in = before + sum;
        if (i < n) {
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                const uint32_t c = v[j];
                v[j] = before;
                before += c;
            }
            memcpy(q, v, sizeof(v));
            reinterpret_cast<uint4*>(counts + i)[0] = q[0], reinterpret_cast<uint4*>(counts + i)[1] = q[1];
        }
        __syncthreads();
        carry = carry_in;
    }
}

// ---- zeros of the rows that no token has -------------------------------------------

constexpr int kFillRows = 32768;  // rows whose presence a CTA knows at a time (4 KB of bits)
// Zeros that take as long as the sort of one CTA, for each of its threads' items (33 us for 16). 16384 x 4096 bf16 into 50257 rows: 105 us,
// with half as much 111, with all of them beside the sort 109.
constexpr int64_t kFillBytes = 15 << 20;

// The rows [r0, r1) without a bit of `present` (bit i: row r0 + i) set to zero by the CTA: a warp takes eight rows, and
// those next to one another as one range.
__device__ __forceinline__ void zero_absent(const EmbedGradArgs& a, int64_t row_bytes, int64_t r0, int64_t r1, const uint32_t* present) {
    for (int64_t r = r0 + (threadIdx.x >> 5) * 8; r < r1; r += (blockDim.x >> 5) * 8) {
        unsigned absent = ~(present[(r - r0) >> 5] >> ((r - r0) & 31)) & 255u;
        if (r1 - r < 8) absent &= (1u << (r1 - r)) - 1u;
        while (absent) {
            const int first = __ffs(absent) - 1, n = __ffs(~(absent >> first)) - 1;
            char* row = static_cast<char*>(a.dtable) + (r + first) * row_bytes;
            zero_bytes(row, row + n * row_bytes);
            absent &= ~(((1u << n) - 1u) << first);
        }
    }
}

// The CTA's share (cta of ctas) of the rows below `rows`, from the ids as they come: every CTA looks at all of them.
__device__ __forceinline__ void fill_unsorted(const EmbedGradArgs& a, int64_t row_bytes, int64_t rows, int64_t cta, int64_t ctas, uint32_t* present) {
    const int64_t begin = rows * cta / ctas, end = rows * (cta + 1) / ctas;
    for (int64_t r0 = begin; r0 < end; r0 += kFillRows) {
        const int64_t r1 = min(r0 + kFillRows, end);
        __syncthreads();
        for (int i = threadIdx.x; i < kFillRows / 32; i += blockDim.x) present[i] = 0;
        __syncthreads();
        const int64_t step = 4 * static_cast<int64_t>(blockDim.x);
        for (int64_t t = threadIdx.x; t < a.tokens; t += step) {
            int64_t id[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) id[j] = t + j * blockDim.x < a.tokens ? __ldg(a.ids + t + j * blockDim.x) : -1;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (id[j] >= r0 && id[j] < r1) atomicOr(&present[(id[j] - r0) >> 5], 1u << ((id[j] - r0) & 31));
        }
        __syncthreads();
        zero_absent(a, row_bytes, r0, r1, present);
    }
}

// How many keys are below `key` (a warp looks at 32 places a step).
__device__ __forceinline__ int64_t keys_below(const uint32_t* keys, int64_t tokens, int64_t key) {
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, hi = tokens;  // below lo keys are smaller, from hi on they are not
    while (lo < hi) {
        const int64_t step = (hi - lo + 31) / 32, t = lo + (lane + 1) * step - 1;
        const int n = __popc(__ballot_sync(kFull, t < hi && keys[t] < key));
        const int64_t next = lo + (n + 1) * step - 1;
        lo += n * step;
        if (next < hi) hi = next;
        if (lo > hi) lo = hi;
    }
    return lo;
}

// Rows whose zeros are written beside the sums, by the first CTAs. (Leaving some to the joining of partial sums gains 0.4 us.)
struct Fill {
    int64_t from, to, row_bytes;
    int ctas;
};
// A CTA's share of them, from the sorted keys.
__device__ __forceinline__ void fill_sorted(const EmbedGradArgs& a, const Fill& f, const uint32_t* keys, uint32_t* present) {
    __shared__ int64_t range[2];
    const int64_t n = f.to - f.from, begin = f.from + n * blockIdx.x / f.ctas, end = f.from + n * (blockIdx.x + 1) / f.ctas;
    for (int64_t r0 = begin; r0 < end; r0 += kFillRows) {
        const int64_t r1 = min(r0 + kFillRows, end);
        __syncthreads();
        for (int i = threadIdx.x; i < kFillRows / 32; i += blockDim.x) present[i] = 0;
        if (threadIdx.x < 64) {
            const int64_t at = keys_below(keys, a.tokens, threadIdx.x < 32 ? r0 : r1);
            if ((threadIdx.x & 31) == 0) range[threadIdx.x >> 5] = at;
        }
        __syncthreads();
        if (range[1] - range[0] <= 4 * (r1 - r0)) {
            for (int64_t t = range[0] + threadIdx.x; t < range[1]; t += blockDim.x) {
                const int64_t bit = keys[t] - r0;
                atomicOr(&present[bit >> 5], 1u << (bit & 31));
            }
        } else {  // many tokens with few ids: each row is looked for
            for (int64_t r = r0 + threadIdx.x; r < r1; r += blockDim.x) {
                int64_t lo = range[0], hi = range[1];
                while (lo < hi) {
                    const int64_t t = (lo + hi) / 2;
                    if (keys[t] < r) lo = t + 1;
                    else hi = t;
                }
                if (lo < range[1] && keys[lo] == r) atomicOr(&present[(r - r0) >> 5], 1u << ((r - r0) & 31));
            }
        }
        __syncthreads();
        zero_absent(a, f.row_bytes, r0, r1, present);
    }
}

// The sort of up to kSortTile tokens by CTA 0 beside the zeros of the first rows by the others; the list of long segments is emptied.
template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads) prepare_kernel(EmbedGradArgs a, int64_t row_bytes, int64_t rows, int bits, uint32_t* keys,
                                                               uint32_t* places, uint32_t* listed) {
    extern __shared__ __align__(16) char raw[];
    pdl_enter();
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) *listed = 0;
        sort_one_tile<ITEMS>(a, bits, keys, places, *reinterpret_cast<SortShared*>(raw));
    } else {
        fill_unsorted(a, row_bytes, rows, static_cast<int64_t>(blockIdx.x) - 1, static_cast<int64_t>(gridDim.x) - 1, reinterpret_cast<uint32_t*>(raw));
    }
}

// ---- sums over segments of equal ids -------------------------------------------------

constexpr int kLong = 2 * kSumTile;  // tokens of the longest segment that one warp sums

struct SumArgs {
    EmbedGradArgs a;
    const uint32_t* keys;
    const uint32_t* places;
    uint32_t* listed;  // how many long segments, then the first token of each
    float* partials;   // [tile][continued, begun][pitch]
    int blocks;        // column blocks of a row
    int pitch;
    Fill fill;
};

// A lane's columns of a row: 16 bytes of it as they lie, and the word after them where rows start elsewhere (WIDE: nowhere).
template <class T, bool WIDE>
struct Piece {
    uint4 lo, hi;
    int shift;
    __device__ __forceinline__ void load(const T* row, int c, int cols) {
        if constexpr (WIDE) {
            if (c < cols) lo = __ldg(reinterpret_cast<const uint4*>(row + c));
        } else {
            const uintptr_t p = reinterpret_cast<uintptr_t>(row + c), end = reinterpret_cast<uintptr_t>(row + cols);
            shift = static_cast<int>(p & 15);
            const uint4* q = reinterpret_cast<const uint4*>(p - shift);
            lo = hi = make_uint4(0, 0, 0, 0);
            if (c < cols) lo = __ldg(q);
            if (c < cols && reinterpret_cast<uintptr_t>(q + 1) < end) hi = __ldg(q + 1);
        }
    }
    __device__ __forceinline__ void add_to(float (&acc)[kLane<T>]) const {
        T e[kLane<T>];
        const uint4 q = WIDE ? lo : shifted(lo, hi, shift);
        memcpy(e, &q, 16);
#pragma unroll
        for (int i = 0; i < kLane<T>; ++i) acc[i] += to_float(e[i]);
    }
};

// dtable[key] (+)= scale acc: a lane's columns from c on, or (not WIDE) turned in shared memory so that neighbouring lanes
// write neighbouring columns.
template <class G, int N, bool WIDE>
__device__ __forceinline__ void write_row(const EmbedGradArgs& a, uint32_t key, int c, const float (&acc)[N], float* turn) {
    G* row = static_cast<G*>(a.dtable) + static_cast<int64_t>(key) * a.cols;
    if constexpr (WIDE) {
        if (c >= a.cols) return;
        float v[N];
        if (a.accumulate) {
            load_floats<G, N>(row + c, v);
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = fmaf(a.scale, acc[k], v[k]);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = a.scale * acc[k];
        }
        store_floats<G, N>(row + c, v);
    } else {
        const int lane = threadIdx.x & 31, c0 = c - lane * N;
        __syncwarp();
#pragma unroll
        for (int k = 0; k < N; ++k) turn[lane * (N + 1) + k] = acc[k];
        __syncwarp();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = 32 * k + lane;
            if (c0 + i >= a.cols) continue;
            const float v = turn[i / N * (N + 1) + i % N];
            row[c0 + i] = from_float<G>(a.accumulate ? fmaf(a.scale, v, to_float(row[c0 + i])) : a.scale * v);
        }
    }
}

template <class T, class G, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2) sum_kernel(SumArgs s) {
    constexpr int N = kLane<T>, kAhead = WIDE ? 16 : 8;  // rows under way
    __shared__ uint32_t shared_words[kFillRows / 32 > kWarps * 32 * (N + 1) ? kFillRows / 32 : kWarps * 32 * (N + 1)];
    pdl_enter();
    const EmbedGradArgs& a = s.a;
    if (static_cast<int>(blockIdx.x) < s.fill.ctas) {
        fill_sorted(a, s.fill, s.keys, shared_words);
        return;
    }
    const int lane = threadIdx.x & 31;
    float* turn = reinterpret_cast<float*>(shared_words) + (threadIdx.x >> 5) * 32 * (N + 1);
    const int64_t units = (a.tokens + kSumTile - 1) / kSumTile * s.blocks;
    for (int64_t unit = (static_cast<int64_t>(blockIdx.x) - s.fill.ctas) * kWarps + (threadIdx.x >> 5); unit < units;
         unit += (static_cast<int64_t>(gridDim.x) - s.fill.ctas) * kWarps) {
        const int64_t tile = unit / s.blocks, t0 = tile * kSumTile;
        const int blk = static_cast<int>(unit - tile * s.blocks), c = (blk * 32 + lane) * N;
        // the keys from 64 tokens before the tile to 64 behind it, the places of those a short segment may have
        uint32_t key[5], place[3];
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            const int64_t t = t0 + 32 * (i - 2) + lane;
            const bool in = t >= 0 && t < a.tokens;
            key[i] = in ? s.keys[t] : kNoKey;
            if (i >= 2) place[i - 2] = in ? s.places[t] : 0;
        }
        const uint32_t mine = key[2], first = __shfl_sync(kFull, mine, 0), before = __shfl_sync(kFull, key[1], 31);
        const uint32_t left = __shfl_up_sync(kFull, mine, 1);
        const unsigned heads = __ballot_sync(kFull, lane == 0 ? mine != before : mine != left);
        const int have = __popc(__ballot_sync(kFull, mine < a.vocab));  // tokens with a row; the others are last
        if (have == 0) continue;
        // tokens right behind the tile that belong to its last segment (64 at most are of interest)
        const uint32_t final = __shfl_sync(kFull, mine, 31);
        const unsigned more1 = __ballot_sync(kFull, key[3] == final), more2 = __ballot_sync(kFull, key[4] == final);
        const int behind = more1 != kFull ? __ffs(~more1) - 1 : more2 != kFull ? 31 + __ffs(~more2) : 64;
        const int next = heads & ~1u ? __ffs(heads & ~1u) - 1 : kSumTile;  // where the first segment ends, if in the tile
        int begin = 0, end = have;
        bool continued = false, long_last = false;
        if (!(heads & 1)) {  // the first segment began before: a long one is summed up to here and in the tile, a short one by its own tile
            const unsigned prev1 = __ballot_sync(kFull, key[1] == first), prev2 = __ballot_sync(kFull, key[0] == first);
            const int ahead = prev1 != kFull ? __clz(~prev1) : prev2 != kFull ? 32 + __clz(~prev2) : 64;
            continued = ahead + (next < kSumTile ? next : kSumTile + behind) > kLong;
            if (!continued) begin = next;
        }
        const unsigned begun = heads & (have == kSumTile ? kFull : (1u << have) - 1u);
        if (have == kSumTile && begun != 0) {
            const int head = 31 - __clz(begun);
            long_last = kSumTile - head + behind > kLong;
            if (!long_last) end = kSumTile + behind;
            else if (blk == 0 && lane == 0) s.listed[1 + atomicAdd(s.listed, 1u)] = static_cast<uint32_t>(t0 + head);
        }
        float acc[N];
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] = 0.0f;
        for (int at = begin; at < end; at += kAhead) {
            Piece<T, WIDE> v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int i = at + j;
                const uint32_t p = __shfl_sync(kFull, i < 32 ? place[0] : i < 64 ? place[1] : place[2], i & 31);
                if (i < end) v[j].load(static_cast<const T*>(a.dy) + static_cast<int64_t>(p) * a.cols, c, a.cols);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int i = at + j;
                if (i >= end) continue;
                v[j].add_to(acc);
                // the last of a segment, or of the tile's part of a long one
                if (i != end - 1 && !(i + 1 < kSumTile && (heads >> (i + 1) & 1))) continue;
                const bool part = (continued && i < next) || (long_last && i == end - 1);
                if (!part) {
                    write_row<G, N, WIDE>(a, __shfl_sync(kFull, mine, min(i, 31)), c, acc, turn);
                } else if (c < a.cols) {
                    store_floats<float, N>(s.partials + (2 * tile + (continued && i < next ? 0 : 1)) * s.pitch + c, acc);
                }
#pragma unroll
                for (int k = 0; k < N; ++k) acc[k] = 0.0f;
            }
        }
    }
}

// The first of the tokens after `from` that has another key (a warp looks at 32 places a step).
__device__ __forceinline__ int64_t segment_end(const uint32_t* keys, int64_t tokens, int64_t from) {
    const uint32_t key = keys[from];
    const int lane = threadIdx.x & 31;
    int64_t lo = from, hi = tokens;  // keys[lo] == key; hi is the end or has another key
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 31) / 32;
        const int64_t t = lo + (lane + 1) * step;
        const unsigned equal = __ballot_sync(kFull, t < hi && keys[t] == key);
        const int n = __popc(equal);  // the first n places have the key
        const int64_t next = lo + static_cast<int64_t>(n + 1) * step;
        lo += n * step;
        if (next < hi) hi = next;
    }
    return hi;
}

// The partial sums of the long segments, added in order: a CTA takes one segment and 256 columns, and each
// of its warps one run of the partials.
template <class G>
__global__ void __launch_bounds__(kThreads) join_kernel(SumArgs s) {
    constexpr int kCols = 256, N = kCols / 32;
    __shared__ float part[kWarps][kCols];
    pdl_enter();
    const EmbedGradArgs& a = s.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, blocks = (a.cols + kCols - 1) / kCols;
    const int64_t items = static_cast<int64_t>(*s.listed) * blocks;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t from = s.listed[1 + item / blocks];
        const int c0 = static_cast<int>(item % blocks) * kCols, c = c0 + lane * N;
        const int64_t end = segment_end(s.keys, a.tokens, from);
        const int64_t first = from / kSumTile, count = (end - 1) / kSumTile - first + 1;
        const int64_t b = count * warp / kWarps, e = count * (warp + 1) / kWarps;
        float acc[N];
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] = 0.0f;
        if (c < a.cols) {
#pragma unroll 8
            for (int64_t i = b; i < e; ++i) {
                float v[N];
                load_floats<float, N>(s.partials + (2 * (first + i) + (i == 0 ? 1 : 0)) * s.pitch + c, v);
#pragma unroll
                for (int k = 0; k < N; ++k) acc[k] += v[k];
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) part[warp][lane * N + k] = acc[k];
        __syncthreads();
        G* row = static_cast<G*>(a.dtable) + static_cast<int64_t>(s.keys[from]) * a.cols;
        for (int i = threadIdx.x; i < kCols && c0 + i < a.cols; i += kThreads) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += part[w][i];
            row[c0 + i] = from_float<G>(a.accumulate ? fmaf(a.scale, sum, to_float(row[c0 + i])) : a.scale * sum);
        }
    }
}

// ---- launches ---------------------------------------------------------------------

// Lanes take 16 bytes where every row starts on 16 bytes.
bool wide(const void* p, int64_t row_bytes) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row_bytes % 16 == 0; }

template <class T>
cudaError_t embed(const EmbedArgs& a, cudaStream_t stream) {
    const int64_t row = a.cols * static_cast<int64_t>(sizeof(T));
    const bool aligned = wide(a.table, row) && wide(a.out, row);
    if (aligned && row < 1024) {
        const int64_t ctas = std::min<int64_t>(ceil_div(a.tokens * (row / 16), 4 * kThreads), 1 << 20);
        return launch_dependent(embed_short_kernel<T>, dim3(static_cast<unsigned>(ctas)), kThreads, 0, 1, stream, a);
    }
    const bool floats = sizeof(T) == 4 && !aligned;
    const int chunks = static_cast<int>(ceil_div(row, floats ? 1024 : 2048));
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(ceil_div(a.tokens * chunks, kWarps), 1 << 20)));
    if (aligned) return launch_dependent(embed_kernel<T>, grid, kThreads, 0, 1, stream, a, chunks);
    if constexpr (sizeof(T) == 4) return launch_dependent(embed_floats_kernel, grid, kThreads, 0, 1, stream, a, chunks);
    else return launch_dependent(embed_odd_kernel<T>, grid, kThreads, 0, 1, stream, a, chunks);
}

template <class T, class G, bool WIDE>
cudaError_t sums(const SumArgs& s0, cudaStream_t stream) {
    SumArgs s = s0;
    s.blocks = static_cast<int>(ceil_div(s.a.cols, 32 * kLane<T>));
    const int64_t ctas = s.fill.ctas + std::min<int64_t>(ceil_div(ceil_div(s.a.tokens, kSumTile) * s.blocks, kWarps), 1 << 20);
    const cudaError_t e = launch_dependent(sum_kernel<T, G, WIDE>, dim3(static_cast<unsigned>(ctas)), kThreads, 0, 1, stream, s);
    if (e != cudaSuccess || s.a.tokens <= kLong) return e;  // no segment can be long
    const int64_t most = std::min<int64_t>(s.a.tokens / (kLong + 1) * ceil_div(s.a.cols, 256), 1024);
    return launch_dependent(join_kernel<G>, dim3(static_cast<unsigned>(most)), kThreads, 0, 1, stream, s);
}

template <class T, class G>
cudaError_t sums_of(const SumArgs& s, cudaStream_t stream) {
    const EmbedGradArgs& a = s.a;
    if (wide(a.dy, a.cols * static_cast<int64_t>(sizeof(T))) && wide(a.dtable, a.cols * static_cast<int64_t>(sizeof(G))))
        return sums<T, G, true>(s, stream);
    return sums<T, G, false>(s, stream);
}

template <int ITEMS>
cudaError_t prepare(const EmbedGradArgs& a, int64_t row, int64_t rows, int64_t fill, int bits, uint32_t* keys, uint32_t* places, uint32_t* listed,
                    cudaStream_t stream) {
    if (!resident_ctas(reinterpret_cast<const void*>(prepare_kernel<ITEMS>), kSortThreads, sizeof(SortShared))) return cudaErrorInvalidConfiguration;
    return launch_dependent(prepare_kernel<ITEMS>, dim3(static_cast<unsigned>(1 + fill)), kSortThreads, sizeof(SortShared), 1, stream, a, row, rows,
                            bits, keys, places, listed);
}

}  // namespace vocab

using namespace vocab;

cudaError_t launch_embedding(int dtype, const EmbedArgs& a, cudaStream_t stream) {
    if (dtype == TR_F32) return embed<float>(a, stream);
    return dtype == TR_BF16 ? embed<__nv_bfloat16>(a, stream) : embed<__half>(a, stream);
}

cudaError_t launch_embedding_backward(int dtype, int grad_dtype, const EmbedGradArgs& a, cudaStream_t stream) {
    const EmbedGradPlan p(a.tokens, a.cols);
    auto at = [&](size_t offset) { return reinterpret_cast<uint32_t*>(a.ws + offset); };
    int bits = 0;
    while (a.vocab >> bits) ++bits;
    const int64_t row = static_cast<int64_t>(a.cols) * (grad_dtype == TR_F32 ? 4 : 2);
    // (its shared memory makes that one CTA an SM)
    const int sms = resident_ctas(reinterpret_cast<const void*>(prepare_kernel<kSortItems>), kSortThreads, sizeof(SortShared));
    if (sms == 0) return cudaErrorInvalidConfiguration;
    int side = 0;
    int64_t filled = 0;  // rows whose zeros are written beside the sort
    cudaError_t e = cudaSuccess;
    if (p.sort_tiles == 1) {
        int items = 1;
        while (items * kSortThreads < a.tokens) items *= 2;
        if (!a.accumulate) filled = std::min<int64_t>(a.vocab, ceil_div(items * kFillBytes, row));
        const int64_t fill = filled > 0 ? std::min<int64_t>(sms - 1, filled) : 0;
        const auto run = items == 1   ? prepare<1>
                         : items == 2 ? prepare<2>
                         : items == 4 ? prepare<4>
                         : items == 8 ? prepare<8>
                                      : prepare<kSortItems>;
        e = run(a, row, filled, fill, bits, at(p.keys[0]), at(p.places[0]), at(p.listed), stream);
    } else {
        const dim3 grid(static_cast<unsigned>(p.sort_tiles));
        for (int shift = 0; shift < bits && e == cudaSuccess; shift += 8) {
            SortPass pass{shift ? at(p.keys[side]) : nullptr, shift ? at(p.places[side]) : nullptr, at(p.keys[side ^ 1]),
                          at(p.places[side ^ 1]), at(p.counts), at(p.listed), p.sort_tiles, shift};
            e = launch_dependent(sort_pass_kernel<false>, grid, kSortThreads, 0, 1, stream, a, pass);
            if (e == cudaSuccess) e = launch_dependent(sort_scan_kernel, dim3(1), kSortThreads, 0, 1, stream, at(p.counts), p.sort_tiles);
            if (e == cudaSuccess) e = launch_dependent(sort_pass_kernel<true>, grid, kSortThreads, 0, 1, stream, a, pass);
            side ^= 1;
        }
    }
    if (e != cudaSuccess) return e;
    const int64_t left = a.accumulate ? 0 : a.vocab - filled;
    const Fill fill{a.vocab - left, a.vocab, row, static_cast<int>(std::min<int64_t>(2 * sms, left))};
    const SumArgs s{a, at(p.keys[side]), at(p.places[side]), at(p.listed), reinterpret_cast<float*>(a.ws + p.partials), 0,
                    static_cast<int>(round_up(a.cols, 8)), fill};
    if (dtype == TR_F32) return sums_of<float, float>(s, stream);
    if (dtype == TR_BF16)
        return grad_dtype == TR_F32 ? sums_of<__nv_bfloat16, float>(s, stream) : sums_of<__nv_bfloat16, __nv_bfloat16>(s, stream);
    return grad_dtype == TR_F32 ? sums_of<__half, float>(s, stream) : sums_of<__half, __half>(s, stream);
}

}  // namespace tr
