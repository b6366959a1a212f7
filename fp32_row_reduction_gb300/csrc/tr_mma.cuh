// Matrix products of 16-bit tiles on the tensor cores: one tile of 256 x (up to 256) by a pair of CTAs.
//
// A cluster of two CTAs computes C = A B^T for 256 rows of A and `width` rows of B (columns of C), summed over the depth in
// blocks of 64. Each CTA brings 128 rows of A and half of B's rows to its shared memory by TMA; one thread of the pair's first CTA
// issues the products for both, and each CTA finds its 128 rows of C, in binary32, in its own tensor memory, where two tiles have
// room: one is written out while the next is summed. An operand lies in memory either with its depth contiguous (rows of 64
// elements are 128 bytes of a 128-byte swizzle) or with its rows contiguous (64 rows of each depth are 128 bytes).
//
// Warp 0 copies, warp 1 issues the products, the others (kOutWarps) write out. The first two run as whole warps, with one lane elected
// at each instruction: the compiler then keeps descriptors and counters in uniform registers. As a single thread, with those
// moved there for each instruction, the second fell behind the tensor cores (574 cycles for a block of 256 x 256 x 64 instead of
// 513, of which the products take 512). Every wait is bounded: one that gives up
// is recorded in the device error word, ends the waits of both CTAs, and makes what is written from then on NaN; the copies and products
// under way are waited for (again bounded) before the pair frees its tensor memory and ends.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "tr_device.cuh"
#include "tr_internal.h"

namespace tr {
namespace mma {

constexpr int kDepth = 64;        // elements of the depth in a block: 128 bytes
constexpr int kRows = 128;        // of A in one CTA
constexpr int kMaxWidth = 256;    // rows of B, both CTAs
constexpr int kStageBytes = (kRows + kMaxWidth / 2) * 128;
constexpr int kStages = 6;
constexpr int kOutWarps = 8;      // two for each quarter of the 128 rows
constexpr int kThreads = 32 * (2 + kOutWarps);
constexpr int kOutBytes = 4096;   // an output warp's room: 32 rows of 128 bytes
constexpr int kSmem = 1024 + kStages * kStageBytes + kOutWarps * kOutBytes;
constexpr int kColumns = 512;     // of tensor memory: two tiles
constexpr long long kLimitNs = 2000000000, kLateNs = 100000000, kTestNs = 1000000;

__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void expect_bytes(uint64_t* bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_addr(bar)),
        "r"(bytes)
        : "memory");
}
__device__ __forceinline__ void arrive_in(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// A box of a tensor map to this CTA's shared memory, its bytes counted on a barrier of the pair.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t what, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(what), "r"(add)
        : "memory");
}
// The products issued so far arrive at this barrier of both CTAs when they are done.
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 32 columns of this warp's 32 rows, a row to a lane.
__device__ __forceinline__ void load_columns(uint32_t addr, float* v) {
    uint32_t r[32];
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 8 columns added to sums that are kept in registers.
__device__ __forceinline__ void add_columns(uint32_t addr, float* v) {
    uint32_t r[8];
    __syncwarp();
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += __uint_as_float(r[i]);
}

// A part's first n of (up to) 128 columns added to sums in registers.
__device__ __forceinline__ void add_part(uint32_t addr, int n, float (&sum)[128]) {
#pragma unroll
    for (int c = 0; c < 128; c += 8)
        if (c < n) add_columns(addr + c, sum + c);
}
// The same where the first part is taken as it is.
__device__ __forceinline__ void take_part(uint32_t addr, int n, bool begun, float (&sum)[128]) {
    if (begun) return add_part(addr, n, sum);
#pragma unroll
    for (int c = 0; c < 128; c += 32)
        if (c < n) load_columns(addr + c, sum + c);
}

// 32 columns of this warp's 32 rows, written.
__device__ __forceinline__ void put_columns(uint32_t addr, const float* v) {
    __syncwarp();
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]),
        "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]),
        "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]),
        "f"(v[31])
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// An output warp's room: 32 rows of 128 bytes in a 128-byte swizzle, on their way to a box of a tensor map.
struct OutBox {
    uint32_t at;
    // once the box that was sent before has been read
    __device__ __forceinline__ void clear() const {
        if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
    }
    // 16-byte word j of the lane's row
    __device__ __forceinline__ void put(int j, uint32_t a, uint32_t b, uint32_t c, uint32_t d) const {
        const int lane = threadIdx.x & 31;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + lane * 128 + ((j ^ (lane & 7)) << 4)), "r"(a), "r"(b), "r"(c), "r"(d)
                     : "memory");
    }
    __device__ __forceinline__ void send(const CUtensorMap* map, int x, int y) const {
        fence_proxy_async_smem();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map), "r"(at), "r"(x), "r"(y) : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
    }
    __device__ __forceinline__ static void finish() {
        if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
};

// Shared-memory descriptor of an operand's block. Depth contiguous: groups of 8 rows are 1024 bytes apart. Rows
// contiguous: groups of 8 depths are 1024 bytes apart, and groups of 64 rows a box of 64 depths.
template <bool ROWS_CONTIGUOUS>
__device__ __forceinline__ uint64_t block_of(uint32_t addr) {
    constexpr uint64_t leading = ROWS_CONTIGUOUS ? kDepth * 128 / 16 : 1, stride = 1024 / 16;
    return (addr >> 4) | leading << 16 | stride << 32 | uint64_t{1} << 46 | uint64_t{2} << 61;
}
// Encoded distance of the next 16 elements of the depth.
template <bool ROWS_CONTIGUOUS>
constexpr uint64_t kNext16 = (ROWS_CONTIGUOUS ? 16 * 128 : 32) / 16;

// The operands of one kind of products, and whether their rows (not their depth) are contiguous in memory. (That has to be known when
// the kernel is compiled: with layouts chosen as it runs, the threads that copy and issue fall behind the tensor
// cores, and the gradients of 8192 x 4096 x 50257 take 5.5 ms instead of 4.9.)
template <bool A_ROWS, bool B_ROWS>
struct Operands {
    static constexpr bool kA = A_ROWS, kB = B_ROWS;
    const CUtensorMap* a;
    const CUtensorMap* b;
    // A of two terms, the second one `second` elements behind the first in each row in memory: its blocks follow those of the first, `blocks` of
    // them, and meet the same B.
    int blocks = 1 << 30;
    int second = 0;
};
// How many rows of A there are at most when all are in one tile (else 256). Rows of a box that lie outside the tensor are
// filled with zeros slowly (one row of hidden in boxes of 128: 122 us instead of 73), so boxes are as high as the rows need,
// and the second CTA copies none when the first has them all: what the products read there instead gives rows of C that nobody takes.
struct Boxes {
    int rows;     // of a box of A, where its depth is contiguous
    bool second;  // whether the second CTA has rows
};
inline Boxes boxes_for(int64_t rows) {
    return Boxes{rows >= kRows ? kRows : static_cast<int>((rows + 7) / 8 * 8), rows > kRows};
}

// What the launch needs apart from the operands.
struct Limits {
    unsigned* err;
    int debug;
};

struct Shared {
    uint64_t full[kStages], empty[kStages], done[2], room[2], never;
    uint32_t columns;
    int dead;
};

// The pair's waits: bounded, and over at once when either CTA has given up.
struct Waits {
    Shared& s;
    Limits lim;
    __device__ __forceinline__ bool dead() const { return *reinterpret_cast<volatile int*>(&s.dead) != 0; }
    __device__ __forceinline__ void die() const {
        if (lim.err) atomicOr(lim.err, kErrWaitTimeout);
        const uint32_t a = smem_addr(&s.dead);
#pragma unroll
        for (uint32_t r = 0; r < 2; ++r) asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(in_cta(a, r)), "r"(1) : "memory");
    }
    // All lanes of a warp wait, and have the same answer. Between two tries the clock is read, which takes long, and it is as well:
    // looking again and again takes shared-memory bandwidth from the products.
    __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
        if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
        const unsigned long long t0 = global_ns();
        while (!__any_sync(kFull, dead())) {
            if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
            if (static_cast<long long>(global_ns() - t0) > kLimitNs) die();
        }
        return false;
    }
};

// An output warp's next tile, or part of one: its place in tensor memory, and how often that place was used.
struct Slot {
    uint32_t number = 0, phase = 0;
    // waits for it; false: after a wait that gave up
    __device__ __forceinline__ bool arrived(const Waits& w) const {
        const bool ok = w.wait(&w.s.done[number], phase) && !__any_sync(kFull, w.dead());
        fence_after();
        return ok;
    }
    // this warp's rows
    __device__ __forceinline__ uint32_t columns(uint32_t all) const { return all + number * kMaxWidth + (threadIdx.x >> 5 & 3) * (32u << 16); }
    // gives the place back
    __device__ __forceinline__ void release(const Waits& w) const {
        fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) arrive_in(in_cta(smem_addr(&w.s.room[number]), 0));
    }
    __device__ __forceinline__ void next() {
        if (++number == 2) number = 0, phase ^= 1;
    }
};

// a / b of numbers that are nearly always below 2^32 (a division of 64 bits takes several times as long).
__device__ __forceinline__ int64_t over(int64_t a, int64_t b) {
    return (a | b) >> 32 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// One unit of work: which tile, and which blocks of the depth.
struct Unit {
    int kind;        // of the products of a launch: 0 or 1
    int m, n;        // first row of A, first row of B
    int begin, end;  // blocks of the depth (equal: the tile is zero)
    int split;
};
// The tiles of one kind of products: in groups of sixteen rows of tiles (what the pairs read at one time is then a little of A
// and of B; groups of eight: 8192 x 4096 x 50257 forward 1760 us instead of 1716), each tile's depth in `splits` parts.
struct Tiles {
    int m = 0, n = 0, splits = 1, blocks = 0;
    __device__ __forceinline__ int64_t units() const { return static_cast<int64_t>(m) * n * splits; }
    __device__ __forceinline__ Unit unit(int kind, int64_t i, int width) const {
        constexpr int kGroup = 16;
        const int64_t t = over(i, splits);
        const int split = static_cast<int>(i - t * splits);
        const int64_t in_group = static_cast<int64_t>(kGroup) * n, g = over(t, in_group);
        const int r = static_cast<int>(t - g * in_group), rows = min(kGroup, m - static_cast<int>(g) * kGroup);
        const int64_t from = static_cast<int64_t>(blocks) * split / splits, to = static_cast<int64_t>(blocks) * (split + 1) / splits;
        return Unit{kind, (static_cast<int>(g) * kGroup + r % rows) * 2 * kRows, r / rows * width, static_cast<int>(from), static_cast<int>(to), split};
    }
};
// The work of a launch: products of one or two kinds, in tiles of one width. A pair takes every (number of pairs)-th unit of the first
// kind; the pairs that this leaves one unit short go ahead with as many rounds of the second kind as fill the time, and
// then all take every so-manyth unit of the rest.
struct Work {
    Tiles first, second;
    int width, pair, pairs;
    int64_t each, longer, ahead;  // units of the first kind of every pair; pairs with one more; rounds that the others go ahead
    __device__ __forceinline__ Work(int w, const Tiles& f, const Tiles& s = Tiles{}) : first(f), second(s), width(w) {
        pair = static_cast<int>(blockIdx.x) / 2;
        pairs = static_cast<int>(gridDim.x) / 2;
        each = over(first.units(), pairs);
        longer = first.units() - each * pairs;
        constexpr int kOut = 12;  // blocks whose products take as long as a tile's beginning and end
        const int one = first.blocks / first.splits + kOut, other = second.blocks + kOut;
        ahead = longer > 0 && second.units() > 0 ? (one + other / 2) / other : 0;
    }
    // The pair's unit number `step`; false: there is none.
    __device__ __forceinline__ bool unit(int64_t step, Unit* u) const {
        const int64_t mine = each + (pair < longer ? 1 : 0);
        if (step < mine) {
            *u = first.unit(0, pair + step * pairs, width);
            return true;
        }
        int64_t i = step - mine;
        const int64_t others = pairs - longer;
        if (pair >= longer && i < ahead) i = i * others + (pair - longer);
        else i = ahead * others + (pair >= longer ? i - ahead : i) * pairs + pair;
        if (i >= second.units()) return false;
        *u = second.unit(1, i, width);
        return true;
    }
};

// How a tile's sums reach the caller of run(): summed over the whole depth, or in parts of so many blocks, because the tensor cores round their
// sums toward zero, an error that grows with the length of a sum. Parts are given to the caller one after another (kEach), or added in registers and put
// back into tensor memory, as if there had been one (kJoined).
enum Parts { kWhole, kEach, kJoined };

// The products of a CTA pair: plan() gives the work, once what earlier kernels wrote can be read; o0 and o1 are the operands of the two
// kinds; `part`: blocks of the depth in a part. out(unit, row, half, first, last,
// tensor address, ok, box, begun, whole, release) takes the columns [first, last) of one row a lane, and calls release() when it has
// read the tensor memory; ok: the sums are there (false: after a wait that gave up); box: the warp's room in
// shared memory; begun: earlier parts have come; whole: the last one.
template <Parts PARTS, class O0, class O1, class Plan, class Out>
__device__ __forceinline__ void run(const O0& o0, const O1& o1, const Boxes& boxes, uint32_t type_bits, const Limits& lim, int part, Plan&& plan, Out&& out) {
    extern __shared__ __align__(16) char raw[];
    __shared__ Shared s;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    // (the same in all lanes, which the compiler knows of a shuffle)
    const int warp = __shfl_sync(kFull, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();
    const Waits waits{s, lim};
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.done[i], 1);
            mbar_init(&s.room[i], 2 * kOutWarps);
        }
        mbar_init(&s.never, 1);
        s.dead = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s.columns)), "r"(kColumns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    // Rows of A that no copy brings are zeros: numbers left there by other kernels would cost power (48 rows of
    // hidden: 97 us instead of 90).
    if (boxes.rows < kRows || !boxes.second) {
        const int from = rank == 0 || boxes.second ? boxes.rows * 8 : 0, words = kRows * 8;  // of 16 bytes
        for (int i = threadIdx.x; i < kStages * words; i += kThreads)
            if (i % words >= from)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(base + i / words * kStageBytes + i % words * 16), "r"(0) : "memory");
        fence_proxy_async_smem();
    }
    fence_before();
    __syncthreads();
    cluster_barrier();
    fence_after();
    const uint32_t columns = s.columns;
    pdl_enter();

    const Work work = plan();
    const int width = work.width;
    int next_stage = 0;  // of the copying warp: where the next block goes, its phase, and how many went before
    uint32_t next_phase = 0, issued = 0;
    if (warp == 0) {
        const uint32_t half = width / 2;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        Unit u{};
        const auto copy = [&](const auto& o) {
            using O = std::decay_t<decltype(o)>;
            const int m = u.m + rank * kRows, n = u.n + rank * half;
            const uint32_t bytes = 128 * (width + (O::kA ? 2 * kRows : boxes.rows * (boxes.second ? 2 : 1)));  // of both CTAs
            for (int k = u.begin; k < u.end; ++k) {
                ok = waits.wait(&s.empty[stage], phase ^ 1);
                if (!ok) break;
                const uint32_t bar = in_cta(smem_addr(&s.full[stage]), 0);
                const uint32_t to_a = base + stage * kStageBytes, to_b = to_a + kRows * 128;
                const bool again = k >= o.blocks;
                const int d = (again ? k - o.blocks : k) * kDepth, a0 = again ? o.second : 0;
                if (rank == 0) expect_bytes(&s.full[stage], bytes);
                if constexpr (O::kA) {
#pragma unroll
                    for (int j = 0; j < kRows / 64; ++j) copy_box(to_a + j * kDepth * 128, o.a, a0 + m + 64 * j, d, bar);
                } else if (rank == 0 || boxes.second) {
                    copy_box(to_a, o.a, a0 + d, m, bar);
                }
                if constexpr (O::kB) {
                    for (uint32_t j = 0; j < half / 64; ++j) copy_box(to_b + j * kDepth * 128, o.b, n + 64 * j, d, bar);
                } else {
                    copy_box(to_b, o.b, d, n, bar);
                }
                ++issued;
                if (++stage == kStages) stage = 0, phase ^= 1;
            }
        };
        for (int64_t i = 0; ok && work.unit(i, &u); ++i) {
            if (u.kind) copy(o1);
            else copy(o0);
        }
        pdl_release();
        next_stage = stage;
        next_phase = phase;
        // Every product's arrival at `empty` reaches the shared memory of both CTAs, and those of the last blocks, which no later copy
        // waits for, may come after that at `done`: each CTA waits for its own, as if kStages more blocks were to be copied, before either may end.
        for (int j = 0; ok && j < kStages; ++j) {
            ok = waits.wait(&s.empty[stage], phase ^ 1);
            if (++stage == kStages) stage = 0, phase ^= 1;
        }
    } else if (warp == 1) {
        if (rank == 0) {
            int stage = 0;
            uint32_t phase = 0, slot = 0, slot_phase = 0;
            bool ok = true;
            if ((lim.debug & kDebugForceTimeout) && blockIdx.x == 0) mbar_wait_bounded(&s.never, 0, kTestNs, lim.err);
            Unit u{};
            const auto multiply = [&](auto&& o) {
                using O = std::decay_t<decltype(o)>;
                // kind::f16: binary32 sums; the operands' type and layouts, width / 8 and 256 / 16
                const uint32_t what = 1u << 4 | type_bits << 7 | type_bits << 10 | (O::kA ? 1u << 15 : 0) | (O::kB ? 1u << 16 : 0) |
                                      static_cast<uint32_t>(width / 8) << 17 | (2 * kRows / 16) << 24;
                int k = u.begin;
                do {
                    const int from = k, to = PARTS != kWhole ? min(k + part, u.end) : u.end;
                    ok = waits.wait(&s.room[slot], slot_phase ^ 1);
                    if (!ok) return;
                    fence_after();
                    const uint32_t d = columns + slot * kMaxWidth;
                    for (; k < to; ++k) {
                        if (lim.debug & kDebugExpireCopies) waits.die(), ok = false;
                        else ok = waits.wait(&s.full[stage], phase);
                        if (!ok) return;
                        fence_after();
                        const uint32_t at = base + stage * kStageBytes;
                        const uint64_t da = block_of<O::kA>(at), db = block_of<O::kB>(at + kRows * 128);
#pragma unroll
                        for (int j = 0; j < kDepth / 16; ++j)
                            product(d, da + j * kNext16<O::kA>, db + j * kNext16<O::kB>, what, k > from || j > 0);
                        commit(smem_addr(&s.empty[stage]));
                        if (++stage == kStages) stage = 0, phase ^= 1;
                    }
                    commit(smem_addr(&s.done[slot]));
                    if (++slot == 2) slot = 0, slot_phase ^= 1;
                } while (k < u.end);
            };
            for (int64_t i = 0; ok && work.unit(i, &u); ++i) {
                if (u.kind) multiply(o1);
                else multiply(o0);
            }
            if (!ok) {  // the products under way
                commit(smem_addr(&s.never));
                mbar_wait_bounded(&s.never, 0, kLateNs, lim.err);
            }
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const int first = half * (width / 2), last = half ? width : width / 2;
        const OutBox box{base + kStages * kStageBytes + (warp - 2) * kOutBytes};
        Slot slot;
        Unit u;
        for (int64_t i = 0; work.unit(i, &u); ++i) {
            const int row = u.m + static_cast<int>(rank) * kRows + quarter * 32 + lane;
            int k = u.begin;
            bool ok = true;
            if (PARTS == kJoined && u.end - k > part) {
                float sum[128];
#pragma unroll
                for (int c = 0; c < 128; ++c) sum[c] = 0.0f;
                for (;; k += part) {
                    ok = slot.arrived(waits) && ok;
                    add_part(slot.columns(columns) + first, last - first, sum);
                    if (u.end - k <= part) break;
                    slot.release(waits);
                    slot.next();
                }
#pragma unroll
                for (int c = 0; c < 128; c += 32)
                    if (c < last - first) put_columns(slot.columns(columns) + first + c, sum + c);
            }
            do {
                const bool begun = PARTS == kEach && k > u.begin;
                k = PARTS == kEach ? min(k + part, u.end) : u.end;
                ok = slot.arrived(waits) && ok;
                out(u, row, half, first, last, slot.columns(columns), ok, box, begun, k >= u.end, [&] { slot.release(waits); });
                slot.next();
            } while (PARTS == kEach && k < u.end);
        }
        OutBox::finish();
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    cluster_barrier();  // with every wait ended well, nothing of either CTA arrives at the other any more
    if (waits.dead()) {
        // After a wait that gave up: blocks may have been copied that no product waited for. Those of both CTAs count on the first one's
        // barriers; what the second began beyond them is given the time.
        if (warp == 0 && rank == 0) {
            for (int j = 0; j < kStages && issued > 0; ++j, --issued) {
                if (next_stage == 0) next_phase ^= 1;
                next_stage = next_stage == 0 ? kStages - 1 : next_stage - 1;
                mbar_wait_bounded(&s.full[next_stage], next_phase, kLateNs, lim.err);
            }
        }
        const unsigned long long t0 = global_ns();
        while (static_cast<long long>(global_ns() - t0) < kTestNs) __nanosleep(1000);
        __syncthreads();
        cluster_barrier();
    }
    fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(columns), "r"(kColumns) : "memory");
}

}  // namespace mma
}  // namespace tr
