// Embedding lookup and its gradient by sorted tokens.
//
// Forward: out[t] = scale table[ids[t]]. A warp takes 2 KB of a row, four 16-byte loads under way together.
//
// Backward: dtable[v] = scale (the sum of dy[t] over the tokens t with ids[t] = v). The tokens are sorted
// by id with a stable radix sort, so that a row's terms come in the order of the tokens and the sums
// repeat bit for bit without atomics. Meanwhile the other CTAs write the zeros of rows that no
// token has: each finds the ids of its own rows in the list. Then a warp sums the rows whose segment starts
// in its 32 sorted tokens, 512 bytes of columns wide, in binary32. Segments longer than 64 tokens
// are cut at the tiles' borders into partial sums, which a last kernel adds in order, so one frequent token
// costs no more than many rare ones.
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

template <class T, int N>
__global__ void __launch_bounds__(kThreads) embed_kernel(EmbedArgs a, int chunks) {
    pdl_enter();
    constexpr int kUnroll = N == 1 ? 8 : 4;
    constexpr int kStep = 32 * N;
    const int lane = threadIdx.x & 31;
    const T* table = static_cast<const T*>(a.table);
    T* out = static_cast<T*>(a.out);
    const int64_t items = a.tokens * chunks;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < items;
         i += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t token = i / chunks;
        const int first = static_cast<int>(i - token * chunks) * (kUnroll * kStep) + lane * N;
        const int64_t id = __ldg(a.ids + token);
        const bool inside = id >= 0 && id < a.vocab;
        const T* src = table + (inside ? id : 0) * a.cols;
        T* dst = out + token * a.cols;
        float v[kUnroll][N];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int c = first + j * kStep;
            if (inside && c < a.cols) load_floats<T, N>(src + c, v[j]);
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int c = first + j * kStep;
#pragma unroll
            for (int k = 0; k < N; ++k) v[j][k] = inside ? a.scale * v[j][k] : 0.0f;
            if (c < a.cols) store_floats<T, N>(dst + c, v[j]);
        }
    }
}

// ---- the sort ----------------------------------------------------------------------

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortItems = kSortTile / kSortThreads;
constexpr uint32_t kNoKey = 0xffffffffu;  // beyond every id: the places after the last token

// Shared memory of a sorting CTA.
struct SortShared {
    uint32_t hist[kSortWarps][kSortBins];
    uint32_t base[kSortBins];
    uint32_t key[kSortTile];
    uint16_t place[kSortTile];
};

// A token's key: its id, or `vocab` (behind every id) when that is outside the table.
__device__ __forceinline__ uint32_t key_of(const EmbedGradArgs& a, int64_t t) {
    const int64_t id = __ldg(a.ids + t);
    return static_cast<uint32_t>(id >= 0 && id < a.vocab ? id : a.vocab);
}

// Item i of a thread: a warp's items are 512 consecutive ones.
__device__ __forceinline__ int item_of(int i) {
    return (threadIdx.x >> 5) * (32 * kSortItems) + i * 32 + (threadIdx.x & 31);
}

// rank[i] = how many items of the tile that come before item i have its digit, once base is added:
// s.hist[w][d] becomes the count of digit d in the warps before w, and `count` (thread d < 256) the tile's
// count of digit d. Begins and ends with a barrier.
__device__ __forceinline__ uint32_t rank_digits(const uint32_t (&key)[kSortItems], int shift, uint32_t (&rank)[kSortItems],
                                                SortShared& s) {
    const int warp = threadIdx.x >> 5;
    const unsigned before = (1u << (threadIdx.x & 31)) - 1u;
    __syncthreads();
    for (int b = threadIdx.x; b < kSortWarps * kSortBins; b += kSortThreads) (&s.hist[0][0])[b] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
        const uint32_t d = (key[i] >> shift) & (kSortBins - 1);
        const unsigned same = __match_any_sync(kFull, d);
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
    for (int i = 0; i < kSortItems; ++i) rank[i] += s.hist[warp][(key[i] >> shift) & (kSortBins - 1)];
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

// Up to kSortTile tokens sorted by one CTA.
__device__ __forceinline__ void sort_one_tile(const EmbedGradArgs& a, int bits, uint32_t* keys, uint32_t* places,
                                              SortShared& s) {
    __shared__ uint32_t warp_total[kSortBins / 32];
    const int n = static_cast<int>(a.tokens);
    uint32_t key[kSortItems], rank[kSortItems];
    uint16_t place[kSortItems];
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
        const int t = item_of(i);
        key[i] = t < n ? key_of(a, t) : kNoKey;
        place[i] = static_cast<uint16_t>(t);
    }
    for (int shift = 0; shift < bits; shift += 8) {
        const uint32_t count = rank_digits(key, shift, rank, s);
        const uint32_t base = bins_before(count, warp_total);
        if (threadIdx.x < kSortBins) s.base[threadIdx.x] = base;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const uint32_t at = s.base[(key[i] >> shift) & (kSortBins - 1)] + rank[i];
            s.key[at] = key[i];
            s.place[at] = place[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            key[i] = s.key[item_of(i)];
            place[i] = s.place[item_of(i)];
        }
    }
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
        const int t = item_of(i);
        if (t < n) {
            keys[t] = key[i];
            places[t] = place[i];
        }
    }
}

// One pass of a sort over several CTAs: the tiles' counts of each digit, their places, the scatter.
struct SortPass {
    const uint32_t* keys;  // null: the first pass, from the ids
    const uint32_t* places;
    uint32_t* out_keys;
    uint32_t* out_places;
    uint32_t* counts;  // [bin][tile]
    int64_t tiles;
    int shift;
};

template <bool SCATTER>
__global__ void __launch_bounds__(kSortThreads) sort_pass_kernel(EmbedGradArgs a, SortPass p) {
    extern __shared__ __align__(16) char raw[];
    SortShared& s = *reinterpret_cast<SortShared*>(raw);
    pdl_enter();
    const int64_t tile = blockIdx.x;
    uint32_t key[kSortItems], rank[kSortItems];
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
        const int64_t t = tile * kSortTile + item_of(i);
        key[i] = t < a.tokens ? (p.keys ? p.keys[t] : key_of(a, t)) : kNoKey;
    }
    const uint32_t count = rank_digits(key, p.shift, rank, s);
    if constexpr (!SCATTER) {
        if (threadIdx.x < kSortBins) p.counts[threadIdx.x * p.tiles + tile] = count;
    } else {
        if (threadIdx.x < kSortBins) s.base[threadIdx.x] = p.counts[threadIdx.x * p.tiles + tile];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const int64_t t = tile * kSortTile + item_of(i);
            if (t < a.tokens) {
                const uint32_t at = s.base[(key[i] >> p.shift) & (kSortBins - 1)] + rank[i];
                p.out_keys[at] = key[i];
                p.out_places[at] = p.places ? p.places[t] : static_cast<uint32_t>(t);
            }
        }
    }
}

// Where each tile's items of each digit go: the counts' exclusive sums in order of digit and tile. (The last
// tile's missing items have digit 255 and are counted last, so they move nothing.)
__global__ void __launch_bounds__(kSortThreads) sort_scan_kernel(uint32_t* counts, int64_t tiles) {
    __shared__ uint32_t warp_total[kSortWarps], carry_in;
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n = tiles * kSortBins;
    uint32_t carry = 0;
    for (int64_t at = 0; at < n; at += kSortThreads) {
        const int64_t i = at + threadIdx.x;
        const uint32_t v = i < n ? counts[i] : 0;
        uint32_t inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += u;
        }
        if (lane == 31) warp_total[warp] = inc;
        __syncthreads();
        uint32_t before = 0;
        for (int w = 0; w < warp; ++w) before += warp_total[w];
        if (i < n) counts[i] = carry + before + inc - v;
        if (threadIdx.x == kSortThreads - 1) carry_in = carry + before + inc;
        __syncthreads();
        carry = carry_in;
    }
}

// ---- zeros of the rows that no token has -------------------------------------------

constexpr int kFillRows = 32768;  // rows whose presence a CTA knows at a time (4 KB of bits)

__device__ __forceinline__ void fill_rows(const EmbedGradArgs& a, int64_t row_bytes, int64_t cta, int64_t ctas,
                                          uint32_t* present) {
    const int64_t begin = a.vocab * cta / ctas, end = a.vocab * (cta + 1) / ctas;
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
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
        for (int64_t r = r0 + warp; r < r1; r += warps) {
            if (present[(r - r0) >> 5] >> ((r - r0) & 31) & 1) continue;
            char* row = static_cast<char*>(a.dtable) + r * row_bytes;
            zero_bytes(row, row + row_bytes);
        }
    }
}

// The sort of up to kSortTile tokens (CTA 0, when `sort`) beside the zeros (the others); the list of long
// segments is emptied.
__global__ void __launch_bounds__(kSortThreads) prepare_kernel(EmbedGradArgs a, int64_t row_bytes, int sort, int bits,
                                                               uint32_t* keys, uint32_t* places, uint32_t* listed) {
    extern __shared__ __align__(16) char raw[];
    pdl_enter();
    if (blockIdx.x == 0 && threadIdx.x == 0) *listed = 0;
    if (sort && blockIdx.x == 0) {
        sort_one_tile(a, bits, keys, places, *reinterpret_cast<SortShared*>(raw));
    } else if (!a.accumulate) {
        fill_rows(a, row_bytes, static_cast<int64_t>(blockIdx.x) - sort, static_cast<int64_t>(gridDim.x) - sort,
                  reinterpret_cast<uint32_t*>(raw));
    }
}

// ---- sums over segments of equal ids -------------------------------------------------

constexpr int kLong = 2 * kSumTile;  // tokens of the longest segment that one warp sums
constexpr int kAhead = 8;            // rows under way

struct SumArgs {
    EmbedGradArgs a;
    const uint32_t* keys;
    const uint32_t* places;
    uint32_t* listed;  // how many long segments, then the first token of each
    float* partials;   // [tile][continued, begun][pitch]
    int blocks;        // column blocks of a row
    int pitch;
};

// dtable[key] (+)= scale acc, one lane's columns.
template <class G, int N>
__device__ __forceinline__ void write_row(const EmbedGradArgs& a, uint32_t key, int c, const float (&acc)[N]) {
    if (c >= a.cols) return;
    G* p = static_cast<G*>(a.dtable) + static_cast<int64_t>(key) * a.cols + c;
    float v[N];
    if (a.accumulate) {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = to_float(p[k]);
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = fmaf(a.scale, acc[k], v[k]);
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = a.scale * acc[k];
    }
    store_floats<G, N>(p, v);
}

// Columns of a block: 32 lanes of N elements, or of eight single ones.
template <int N>
constexpr int kBlockCols = N == 1 ? 256 : 32 * N;

template <class T, class G, int N>
__global__ void __launch_bounds__(kThreads) sum_kernel(SumArgs s) {
    constexpr int kParts = N == 1 ? 8 : 1;  // single elements: eight columns a lane, 32 apart
    constexpr int kSpan = kSumTile + kLong;
    __shared__ uint32_t key_window[kLong + kSpan + kLong + 1];  // from kLong tokens before the tile
    __shared__ uint32_t place_window[kSpan];
    pdl_enter();
    const EmbedGradArgs& a = s.a;
    const int lane = threadIdx.x & 31;
    const int groups = (s.blocks + kWarps - 1) / kWarps;
    const int64_t tiles = (a.tokens + kSumTile - 1) / kSumTile;
    for (int64_t item = blockIdx.x; item < tiles * groups; item += gridDim.x) {
        const int64_t tile = item / groups, t0 = tile * kSumTile;
        const int blk = static_cast<int>(item - tile * groups) * kWarps + (threadIdx.x >> 5);
        __syncthreads();
        for (int i = threadIdx.x; i < kLong + kSpan + kLong + 1; i += kThreads) {
            const int64_t t = t0 - kLong + i;
            key_window[i] = t >= 0 && t < a.tokens ? s.keys[t] : kNoKey;
            if (i < kSpan) place_window[i] = t0 + i < a.tokens ? s.places[t0 + i] : 0;
        }
        __syncthreads();
        if (blk >= s.blocks) continue;  // (no barrier before the loop's next)
        const uint32_t* keys = key_window + kLong;
        const int have = static_cast<int>(min(static_cast<int64_t>(kSumTile), a.tokens - t0));
        const int c0 = blk * kBlockCols<N> + lane * (N == 1 ? 1 : N);
        // the segment that reaches in from the tile before, if it is long, is this tile's up to its end
        int at = 0;
        bool continued = false;
        if (t0 > 0 && keys[-1] == keys[0]) {
            int first = -1;
            while (first > -kLong && keys[first - 1] == keys[0]) --first;
            continued = keys[first + kLong] == keys[0];
            if (!continued)
                while (at < have && keys[at] == keys[0]) ++at;  // its own tile sums it
        }
        float acc[kParts][N];
#pragma unroll
        for (int q = 0; q < kParts; ++q)
#pragma unroll
            for (int k = 0; k < N; ++k) acc[q][k] = 0.0f;
        // whether the segment at `at` is long
        bool large = continued;
        bool fresh = !continued;  // `at` begins a segment
        int stop = have;          // a short segment that begins in the tile is summed to its end
        while (at < stop) {
            float v[kAhead][kParts][N];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int i = min(at + j, kSpan - 1);
                const bool mine = keys[i] < a.vocab && (i < have || keys[i] == keys[have - 1]);
                const T* row = static_cast<const T*>(a.dy) + static_cast<int64_t>(place_window[i]) * a.cols;
#pragma unroll
                for (int q = 0; q < kParts; ++q) {
                    const int c = c0 + 32 * q;
                    if (mine && c < a.cols) load_floats<T, N>(row + c, v[j][q]);
                }
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (at < stop) {
                    const uint32_t key = keys[at];
                    if (key >= a.vocab) {  // behind the last id: nothing more
                        stop = at;
                    } else {
                        if (fresh) {
                            large = keys[at + kLong] == key;
                            fresh = false;
                            if (large && blk == 0 && lane == 0) s.listed[1 + atomicAdd(s.listed, 1u)] = static_cast<uint32_t>(t0 + at);
                            if (!large)
                                while (keys[stop - 1] == key && keys[stop] == key) ++stop;
                        }
#pragma unroll
                        for (int q = 0; q < kParts; ++q)
#pragma unroll
                            for (int k = 0; k < N; ++k) acc[q][k] += v[j][q][k];
                        ++at;
                        const bool last = keys[at] != key;
                        if (last || (large && at == have)) {
#pragma unroll
                            for (int q = 0; q < kParts; ++q) {
                                const int c = c0 + 32 * q;
                                if (!large) {
                                    write_row<G, N>(a, key, c, acc[q]);
                                } else if (c < a.cols) {
                                    float* p = s.partials + (2 * tile + (continued ? 0 : 1)) * s.pitch + c;
                                    store_floats<float, N>(p, acc[q]);
                                }
#pragma unroll
                                for (int k = 0; k < N; ++k) acc[q][k] = 0.0f;
                            }
                            continued = false;
                            fresh = true;
                        }
                    }
                }
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

// The partial sums of the long segments, added in order: a CTA takes one segment and one block of columns, and each
// of its warps one run of the partials.
template <class G, int N>
__global__ void __launch_bounds__(kThreads) join_kernel(SumArgs s) {
    constexpr int kParts = N == 1 ? 8 : 1;
    __shared__ float part[kWarps][kBlockCols<N>];
    pdl_enter();
    const EmbedGradArgs& a = s.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t items = static_cast<int64_t>(*s.listed) * s.blocks;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t from = s.listed[1 + item / s.blocks];
        const int c0 = static_cast<int>(item % s.blocks) * kBlockCols<N> + lane * (N == 1 ? 1 : N);
        const int64_t end = segment_end(s.keys, a.tokens, from);
        const int64_t first = from / kSumTile, count = (end - 1) / kSumTile - first + 1;
        const int64_t b = count * warp / kWarps, e = count * (warp + 1) / kWarps;
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
            const int c = c0 + 32 * q;
            float acc[N];
#pragma unroll
            for (int k = 0; k < N; ++k) acc[k] = 0.0f;
            if (c < a.cols) {
#pragma unroll 4
                for (int64_t i = b; i < e; ++i) {
                    float v[N];
                    load_floats<float, N>(s.partials + (2 * (first + i) + (i == 0 ? 1 : 0)) * s.pitch + c, v);
#pragma unroll
                    for (int k = 0; k < N; ++k) acc[k] += v[k];
                }
            }
#pragma unroll
            for (int k = 0; k < N; ++k) part[warp][32 * q + lane * (N == 1 ? 1 : N) + k] = acc[k];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < kBlockCols<N>; c += kThreads) {
            float acc[1] = {0.0f};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) acc[0] += part[w][c];
            write_row<G, 1>(a, s.keys[from], static_cast<int>(item % s.blocks) * kBlockCols<N> + c, acc);
        }
    }
}

// ---- launches ---------------------------------------------------------------------

// Lanes take 16 bytes where every row starts on 16 bytes.
bool wide(const void* p, int64_t row_bytes) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row_bytes % 16 == 0; }

template <class T, int N>
cudaError_t embed(const EmbedArgs& a, cudaStream_t stream) {
    constexpr int kChunk = (N == 1 ? 8 : 4) * 32 * N;
    const int chunks = static_cast<int>(ceil_div(a.cols, kChunk));
    const int64_t ctas = std::min<int64_t>(ceil_div(a.tokens * chunks, kWarps), 1 << 20);
    return launch_dependent(embed_kernel<T, N>, dim3(static_cast<unsigned>(ctas)), kThreads, 0, 1, stream, a, chunks);
}

template <class T, class G, int N>
cudaError_t sums(const SumArgs& s0, int64_t sum_tiles, cudaStream_t stream) {
    SumArgs s = s0;
    s.blocks = static_cast<int>(ceil_div(s.a.cols, kBlockCols<N>));
    const int64_t items = sum_tiles * ceil_div(s.blocks, kWarps);
    cudaError_t e = launch_dependent(sum_kernel<T, G, N>, dim3(static_cast<unsigned>(std::min<int64_t>(items, 1 << 20))),
                                     kThreads, 0, 1, stream, s);
    if (e != cudaSuccess || s.a.tokens <= kLong) return e;  // no segment can be long
    const int64_t most = std::min<int64_t>(s.a.tokens / (kLong + 1) * s.blocks, 1024);
    return launch_dependent(join_kernel<G, N>, dim3(static_cast<unsigned>(most)), kThreads, 0, 1, stream, s);
}

template <class T, class G>
cudaError_t sums_of(const SumArgs& s, int64_t sum_tiles, cudaStream_t stream) {
    constexpr int N = 16 / sizeof(T);
    const EmbedGradArgs& a = s.a;
    if (wide(a.dy, a.cols * static_cast<int64_t>(sizeof(T))) && wide(a.dtable, a.cols * static_cast<int64_t>(sizeof(G))))
        return sums<T, G, N>(s, sum_tiles, stream);
    return sums<T, G, 1>(s, sum_tiles, stream);
}

}  // namespace vocab

using namespace vocab;

cudaError_t launch_embedding(int dtype, const EmbedArgs& a, cudaStream_t stream) {
    const int64_t row = static_cast<int64_t>(a.cols) * (dtype == TR_F32 ? 4 : 2);
    const bool w = wide(a.table, row) && wide(a.out, row);
    if (dtype == TR_F32) return w ? embed<float, 4>(a, stream) : embed<float, 1>(a, stream);
    if (dtype == TR_BF16) return w ? embed<__nv_bfloat16, 8>(a, stream) : embed<__nv_bfloat16, 1>(a, stream);
    return w ? embed<__half, 8>(a, stream) : embed<__half, 1>(a, stream);
}

cudaError_t launch_embedding_backward(int dtype, int grad_dtype, const EmbedGradArgs& a, cudaStream_t stream) {
    const EmbedGradPlan p(a.tokens, a.cols);
    auto at = [&](size_t offset) { return reinterpret_cast<uint32_t*>(a.ws + offset); };
    int bits = 0;
    while (a.vocab >> bits) ++bits;
    const int64_t row = static_cast<int64_t>(a.cols) * (grad_dtype == TR_F32 ? 4 : 2);
    const int smem = sizeof(SortShared);
    // one CTA an SM, which the sort's shared memory makes of it
    const int resident = resident_ctas(reinterpret_cast<const void*>(prepare_kernel), kSortThreads, smem);
    if (resident == 0) return cudaErrorInvalidConfiguration;
    const int one = p.sort_tiles == 1 ? 1 : 0;
    const int64_t fill = a.accumulate ? 0 : std::max<int64_t>(1, std::min<int64_t>(resident - one, a.vocab));
    cudaError_t e = launch_dependent(prepare_kernel, dim3(static_cast<unsigned>(std::max<int64_t>(1, one + fill))), kSortThreads,
                                     smem, 1, stream, a, row, one, bits, at(p.keys[0]), at(p.places[0]), at(p.listed));
    int side = 0;
    if (!one) {
        if (!resident_ctas(reinterpret_cast<const void*>(sort_pass_kernel<false>), kSortThreads, smem) ||
            !resident_ctas(reinterpret_cast<const void*>(sort_pass_kernel<true>), kSortThreads, smem))
            return cudaErrorInvalidConfiguration;
        const dim3 grid(static_cast<unsigned>(p.sort_tiles));
        for (int shift = 0; shift < bits && e == cudaSuccess; shift += 8) {
            SortPass pass{shift ? at(p.keys[side]) : nullptr, shift ? at(p.places[side]) : nullptr, at(p.keys[side ^ 1]),
                          at(p.places[side ^ 1]), at(p.counts), p.sort_tiles, shift};
            e = launch_dependent(sort_pass_kernel<false>, grid, kSortThreads, smem, 1, stream, a, pass);
            if (e == cudaSuccess) e = launch_dependent(sort_scan_kernel, dim3(1), kSortThreads, 0, 1, stream, at(p.counts), p.sort_tiles);
            if (e == cudaSuccess) e = launch_dependent(sort_pass_kernel<true>, grid, kSortThreads, smem, 1, stream, a, pass);
            side ^= 1;
        }
    }
    if (e != cudaSuccess) return e;
    const SumArgs s{a, at(p.keys[side]), at(p.places[side]), at(p.listed), reinterpret_cast<float*>(a.ws + p.partials), 0,
                    static_cast<int>(round_up(a.cols, 8))};
    if (dtype == TR_F32) return sums_of<float, float>(s, p.sum_tiles, stream);
    if (dtype == TR_BF16)
        return grad_dtype == TR_F32 ? sums_of<__nv_bfloat16, float>(s, p.sum_tiles, stream)
                                    : sums_of<__nv_bfloat16, __nv_bfloat16>(s, p.sum_tiles, stream);
    return grad_dtype == TR_F32 ? sums_of<__half, float>(s, p.sum_tiles, stream) : sums_of<__half, __half>(s, p.sum_tiles, stream);
}

}  // namespace tr
