// C-ABI of the block norms and of the norms over a list of tensors: argument
// checks on the host, then the launches. No entry point allocates device memory, waits, or
// lets a C++ exception out.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <map>
#include <mutex>
#include <new>
#include <tuple>
#include <vector>

#include "tr.h"
#include "tr_block.h"
#include "tr_internal.h"
#include "tr_launch.h"
#include "tr_list.h"

namespace tr {
namespace {

tr_status fail(tr_status s, const char* where, const char* why) {
    set_last_error(where, why);
    return s;
}
// An error is also cleared from the runtime's last-error slot, which other entry points ask after their own launches.
tr_status cuda_status(cudaError_t e, const char* where) {
    if (e == cudaSuccess) return TR_OK;
    cudaGetLastError();
    return fail(TR_ERR_CUDA, where, cudaGetErrorString(e));
}

size_t element_bytes(int dtype) { return dtype == TR_F32 ? 4 : 2; }

struct Range {
    const void* p;
    size_t bytes;
    size_t align;
    bool overlaps(const Range& o) const {
        if (!p || !o.p || bytes == 0 || o.bytes == 0) return false;
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
        return a < b + o.bytes && b < a + bytes;
    }
    bool misaligned() const { return p && reinterpret_cast<uintptr_t>(p) % align != 0; }
};

// Alignment of every range; no output overlapping an input or another output.
template <size_t I, size_t O>
tr_status check_ranges(const char* where, const Range (&in)[I], const Range (&out)[O]) {
    for (const Range& r : in)
        if (r.misaligned()) return fail(TR_ERR_INVALID_ARG, where, "a misaligned input pointer");
    for (size_t o = 0; o < O; ++o) {
        if (out[o].misaligned()) return fail(TR_ERR_INVALID_ARG, where, "a misaligned output or workspace pointer");
        for (const Range& r : in)
            if (out[o].overlaps(r)) return fail(TR_ERR_INVALID_ARG, where, "an output or the workspace overlaps an input");
        for (size_t q = o + 1; q < O; ++q)
            if (out[o].overlaps(out[q])) return fail(TR_ERR_INVALID_ARG, where, "two outputs (or the workspace) overlap");
    }
    return TR_OK;
}

tr_status check_block(const char* w, int kind, int dtype, int norms, const float* post_w, const float* post_b,
                      const float* gate, int64_t gate_rows, const float* pre_w, const float* pre_b, int64_t rows,
                      int64_t cols, float rs, float bs, float eps, int order) {
    if (kind != TR_NORM_RMS && kind != TR_NORM_LAYER) return fail(TR_ERR_INVALID_ARG, w, "kind must be a tr_norm_kind");
    if (dtype != TR_F32 && dtype != TR_BF16 && dtype != TR_F16)
        return fail(TR_ERR_INVALID_ARG, w, "dtype must be a tr_dtype");
    if (norms < 1 || (norms & ~(TR_BLOCK_POST | TR_BLOCK_PRE)))
        return fail(TR_ERR_INVALID_ARG, w, "norms must be TR_BLOCK_POST, TR_BLOCK_PRE or both");
    if (order < TR_ORDER_UNORDERED_TREE || order > TR_ORDER_FOLD_RIGHT)
        return fail(TR_ERR_INVALID_ARG, w, "order must be one of the tr_order values");
    if (order != TR_ORDER_UNORDERED_TREE)
        return fail(TR_ERR_UNSUPPORTED, w, "the block norms take the unordered policy only");
    if (rows < 0) return fail(TR_ERR_INVALID_ARG, w, "rows must be >= 0");
    if (cols < 1 || cols >= (1 << 24)) return fail(TR_ERR_INVALID_ARG, w, "cols must be in [1, 2^24 - 1]");
    if (rows > INT64_MAX / cols / 4) return fail(TR_ERR_INVALID_ARG, w, "rows * cols too large");
    if (!std::isfinite(eps) || eps < 0.0f) return fail(TR_ERR_INVALID_ARG, w, "eps must be finite and >= 0");
    if (!std::isfinite(rs) || !std::isfinite(bs)) return fail(TR_ERR_INVALID_ARG, w, "the scales must be finite");
    if (gate && (gate_rows < 1 || rows % gate_rows != 0))
        return fail(TR_ERR_INVALID_ARG, w, "gate_rows must divide rows");
    if (!(norms & TR_BLOCK_POST) && (post_w || post_b))
        return fail(TR_ERR_INVALID_ARG, w, "post_w and post_b need TR_BLOCK_POST");
    if (!(norms & TR_BLOCK_PRE) && (pre_w || pre_b))
        return fail(TR_ERR_INVALID_ARG, w, "pre_w and pre_b need TR_BLOCK_PRE");
    if (kind == TR_NORM_RMS && (post_b || pre_b)) return fail(TR_ERR_INVALID_ARG, w, "RMSNorm takes no bias");
    return TR_OK;
}

size_t stats_bytes(int64_t rows) { return static_cast<size_t>(rows) * kBlockStats * sizeof(float); }

size_t backward_bytes(int kind, int64_t rows, int64_t cols) {
    if (rows == 0) return 0;
    return stats_bytes(rows) + static_cast<size_t>(block_slab_limit(rows, cols)) * block_vectors(kind) *
                                   static_cast<size_t>(cols) * sizeof(float);
}

// ---- lists ------------------------------------------------------------------

struct ListCall {
    const void* const* tensors;
    void* const* outs;  // null: read only
    const int64_t* numels;
    const int32_t* dtypes;
    int64_t count;
};

constexpr int64_t kListMaxNumel = 1LL << 42;  // 2^44 bytes: beyond any device, and tile counts stay below 2^31

tr_status check_list(const char* w, const ListCall& l, const void* norm, const void* ws, size_t ws_bytes) {
    if (l.count < 0) return fail(TR_ERR_INVALID_ARG, w, "count must be >= 0");
    if (!norm) return fail(TR_ERR_INVALID_ARG, w, "norm must not be null");
    const Range fixed[2] = {{norm, 4, 4}, {ws, ws_bytes, 16}};
    if (fixed[0].misaligned()) return fail(TR_ERR_INVALID_ARG, w, "norm must be 4-byte aligned");
    if (fixed[1].misaligned()) return fail(TR_ERR_INVALID_ARG, w, "the workspace must be 16-byte aligned");
    if (fixed[0].overlaps(fixed[1])) return fail(TR_ERR_INVALID_ARG, w, "norm overlaps the workspace");
    if (l.count == 0) return TR_OK;
    if (!l.tensors || !l.numels || !l.dtypes) return fail(TR_ERR_INVALID_ARG, w, "the list's arrays must not be null");
    for (int64_t i = 0; i < l.count; ++i) {
        const int d = l.dtypes[i];
        if (d != TR_F32 && d != TR_BF16 && d != TR_F16) return fail(TR_ERR_INVALID_ARG, w, "dtypes must be tr_dtype values");
        const int64_t n = l.numels[i];
        if (n < 0 || n > kListMaxNumel) return fail(TR_ERR_INVALID_ARG, w, "numels must be in [0, 2^42]");
        if (n == 0) continue;
        const size_t b = element_bytes(d);
        const Range in{l.tensors[i], static_cast<size_t>(n) * b, b};
        const Range out{l.outs ? l.outs[i] : nullptr, in.bytes, b};
        if (!in.p || (l.outs && !out.p)) return fail(TR_ERR_INVALID_ARG, w, "a tensor pointer is null");
        if (in.misaligned() || out.misaligned()) return fail(TR_ERR_INVALID_ARG, w, "a tensor is not aligned to its elements");
        for (const Range& f : fixed)
            if (f.overlaps(in) || f.overlaps(out))
                return fail(TR_ERR_INVALID_ARG, w, "norm or the workspace overlaps a tensor");
    }
    return TR_OK;
}

// Written tensors may overlap neither one another nor a tensor of the list that is
// not the same one: after sorting all ranges by start, only a written range can
// make its successor (or be made by its predecessor) a conflict.
tr_status check_written(const char* w, const ListCall& l) {
    struct Span {
        uintptr_t begin, end;
        bool written;
    };
    std::vector<Span> spans;
    spans.reserve(static_cast<size_t>(l.count) * 2);
    for (int64_t i = 0; i < l.count; ++i) {
        if (l.numels[i] == 0) continue;
        const size_t n = static_cast<size_t>(l.numels[i]) * element_bytes(l.dtypes[i]);
        const uintptr_t in = reinterpret_cast<uintptr_t>(l.tensors[i]), out = reinterpret_cast<uintptr_t>(l.outs[i]);
        spans.push_back(Span{out, out + n, true});
        if (in != out) spans.push_back(Span{in, in + n, false});
    }
    auto less = [](const Span& a, const Span& b) { return a.begin < b.begin; };
    if (!std::is_sorted(spans.begin(), spans.end(), less)) std::sort(spans.begin(), spans.end(), less);
    uintptr_t end_any = 0, end_written = 0;  // how far the ranges so far reach
    for (const Span& s : spans) {
        if (s.begin < end_written || (s.written && s.begin < end_any))
            return fail(TR_ERR_INVALID_ARG, w, "a tensor that is written overlaps another tensor of the list");
        end_any = std::max(end_any, s.end);
        if (s.written) end_written = std::max(end_written, s.end);
    }
    return TR_OK;
}

// fn(list) for the list in launches of at most kListMax tensors.
template <class F>
cudaError_t for_launches(const ListCall& c, F&& fn) {
    static thread_local TensorList<kListMax> l;
    l.count = 0;
    l.first[0] = 0;
    for (int64_t i = 0; i < c.count; ++i) {
        if (c.numels[i] == 0) continue;
        const int k = l.count;
        const size_t b = element_bytes(c.dtypes[i]);
        const uint64_t bytes = (reinterpret_cast<uintptr_t>(c.tensors[i]) & 15) + static_cast<uint64_t>(c.numels[i]) * b;
        const uint64_t tiles = (bytes + kListTileBytes - 1) / kListTileBytes;
        if (k == kListMax || (k > 0 && l.first[k] + tiles > UINT32_MAX)) {
            const cudaError_t e = fn(l);
            if (e != cudaSuccess) return e;
            l.count = 0;
            --i;
            continue;
        }
        l.in[k] = static_cast<const char*>(c.tensors[i]);
        l.out[k] = c.outs ? static_cast<char*>(c.outs[i]) : nullptr;
        l.numel[k] = c.numels[i];
        l.dtype[k] = static_cast<uint8_t>(c.dtypes[i]);
        l.first[k + 1] = l.first[k] + static_cast<uint32_t>(tiles);
        l.count = k + 1;
    }
    return l.count > 0 ? fn(l) : cudaSuccess;
}

// A launch more than the count asks for can come of the tile limit: at 2^32 tiles
// (64 TB) a launch, beyond any device's memory, so the workspace holds one launch's
// partials per kListMax tensors and a spare.
size_t norm_bytes(int64_t count) {
    return static_cast<size_t>(list_launches(count) + 1) * kListMaxCtas * sizeof(double);
}

tr_status list_norm(const char* w, int kind, const ListCall& c, float* norm, void* ws, size_t ws_bytes, int* n,
                    cudaStream_t stream) {
    if (kind != TR_TOTAL_L2 && kind != TR_TOTAL_MAX) return fail(TR_ERR_INVALID_ARG, w, "kind must be a tr_total_kind");
    const tr_status s = check_list(w, c, norm, ws, ws_bytes);
    if (s != TR_OK) return s;
    if (!ws || ws_bytes < norm_bytes(c.count))
        return fail(TR_ERR_INVALID_ARG, w, "the workspace is missing or smaller than tr_global_norm_workspace_bytes");
    if (c.outs) {
        const tr_status o = check_written(w, c);
        if (o != TR_OK) return o;
    }
    double* part = static_cast<double*>(ws);
    const int64_t cap = static_cast<int64_t>(norm_bytes(c.count) / sizeof(double));
    *n = 0;
    return cuda_status(for_launches(c, [&](const TensorList<kListMax>& l) {
                           if (*n + kListMaxCtas > cap) return cudaErrorInvalidValue;
                           int ctas = 0;
                           const cudaError_t e = launch_list_norm(kind, l, part + *n, c.outs != nullptr, &ctas, stream);
                           *n += ctas;
                           return e;
                       }), w);
}

tr_status scale_list(const char* w, int kind, const ListCall& c, const double* part, int n, float* norm, bool write,
                     float max_norm, float eps, cudaStream_t stream) {
    return cuda_status(for_launches(c, [&](const TensorList<kListMax>& l) {
                           const cudaError_t e = launch_list_scale(kind, l, part, n, norm, write ? 1 : 0, max_norm, eps, stream);
                           write = false;
                           return e;
                       }), w);
}

tr_status check_clip(const char* w, float max_norm, float eps) {
    if (!(max_norm >= 0.0f)) return fail(TR_ERR_INVALID_ARG, w, "max_norm must be >= 0");
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(TR_ERR_INVALID_ARG, w, "eps must be finite and >= 0");
    return TR_OK;
}

template <class F>
tr_status guarded(const char* w, F&& f) {
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return fail(TR_ERR_UNSUPPORTED, w, "out of host memory");
    } catch (...) {
        return fail(TR_ERR_UNSUPPORTED, w, "an unexpected host error");
    }
}

std::mutex g_launch_mu;
std::map<std::tuple<int, const void*, int, size_t, int>, int> g_resident;
std::map<int, unsigned*> g_error_words;

}  // namespace

bool dependent_launches() {
    static const bool on = [] {
        const char* v = std::getenv("TR_DISABLE_PDL");
        return !(v && v[0] == '1');
    }();
    return on;
}

unsigned* device_error_word() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
    std::lock_guard<std::mutex> lock(g_launch_mu);
    const auto it = g_error_words.find(dev);
    if (it != g_error_words.end()) return it->second;
    void* p = nullptr;
    if (device_error_symbol(&p) != cudaSuccess) return nullptr;
    return g_error_words[dev] = static_cast<unsigned*>(p);
}

int resident_ctas(const void* kernel, int threads, size_t smem, int cluster) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lock(g_launch_mu);
    const auto key = std::make_tuple(dev, kernel, threads, smem, cluster);
    const auto it = g_resident.find(key);
    if (it != g_resident.end()) return it->second;
    int per = 0, sms = 0, optin = 0;
    cudaFuncAttributes fa;
    // the kernel's limit is raised once, as far as the device lets it
    cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kernel);
    if (e == cudaSuccess && smem > 0)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin - static_cast<int>(fa.sharedSizeBytes));
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem);
    int ctas = per * sms;
    if (e == cudaSuccess && cluster > 1) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(cluster));
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = cluster;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
        ctas = clusters * cluster;
    }
    if (e != cudaSuccess) return 0;  // not kept: the launch reports the error
    return g_resident[key] = ctas;
}

}  // namespace tr

using namespace tr;

extern "C" {

tr_status tr_gated_residual_norm(tr_norm_kind kind, tr_dtype dtype, int32_t norms, const void* x, const void* branch,
                                 const float* post_w, const float* post_b, const float* gate, int64_t gate_rows,
                                 const float* pre_w, const float* pre_b, void* h, void* y, int64_t rows, int64_t cols,
                                 float residual_scale, float branch_scale, float eps, tr_order order,
                                 cudaStream_t stream) {
    static const char* w = "gated residual norm";
    tr_status s = check_block(w, kind, dtype, norms, post_w, post_b, gate, gate_rows, pre_w, pre_b, rows, cols,
                              residual_scale, branch_scale, eps, order);
    if (s != TR_OK) return s;
    const bool pre = norms & TR_BLOCK_PRE;
    if (!pre && y) return fail(TR_ERR_INVALID_ARG, w, "y needs TR_BLOCK_PRE");
    if (rows == 0) return TR_OK;
    if (!x || !branch) return fail(TR_ERR_INVALID_ARG, w, "x and branch must not be null");
    if (pre ? !y : !h) return fail(TR_ERR_INVALID_ARG, w, "y (or, without TR_BLOCK_PRE, h) must not be null");
    const size_t eb = element_bytes(dtype), n = static_cast<size_t>(rows) * cols * eb, nc = static_cast<size_t>(cols) * 4;
    const Range in[] = {{x, n, eb}, {branch, n, eb}, {post_w, nc, 4}, {post_b, nc, 4}, {pre_w, nc, 4}, {pre_b, nc, 4},
                        {gate, gate ? nc * static_cast<size_t>(gate_rows) : 0, 4}};
    const Range out[] = {{h, n, eb}, {y, n, eb}};
    s = check_ranges(w, in, out);
    if (s != TR_OK) return s;
    BlockArgs a{x, branch, h, y, post_w, post_b, gate, pre_w, pre_b, rows, gate ? rows / gate_rows : rows,
                static_cast<int>(cols), norms & TR_BLOCK_POST ? 1 : 0, pre ? 1 : 0, residual_scale, branch_scale, eps, nullptr};
    return guarded(w, [&] { return cuda_status(launch_block_forward(kind, dtype, a, stream), w); });
}

tr_status tr_gated_residual_norm_backward_workspace_bytes(tr_norm_kind kind, int64_t rows, int64_t cols, size_t* bytes) {
    static const char* w = "gated residual norm backward workspace";
    if (!bytes) return fail(TR_ERR_INVALID_ARG, w, "bytes must not be null");
    const tr_status s = check_block(w, kind, TR_F32, TR_BLOCK_PRE, nullptr, nullptr, nullptr, 0, nullptr, nullptr, rows,
                                    cols, 1.0f, 1.0f, 0.0f, TR_ORDER_UNORDERED_TREE);
    if (s != TR_OK) return s;
    *bytes = backward_bytes(kind, rows, cols);
    return TR_OK;
}

tr_status tr_gated_residual_norm_backward(tr_norm_kind kind, tr_dtype dtype, int32_t norms, const void* h,
                                          const void* branch, const void* dy, const void* dh, const float* post_w,
                                          const float* post_b, const float* gate, int64_t gate_rows,
                                          const float* pre_w, void* dx, void* dbranch, float* dpost_w, float* dpost_b,
                                          float* dgate, float* dpre_w, float* dpre_b, int64_t rows, int64_t cols,
                                          float residual_scale, float branch_scale, float eps, tr_order order,
                                          void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    static const char* w = "gated residual norm backward";
    tr_status s = check_block(w, kind, dtype, norms, post_w, post_b, gate, gate_rows, pre_w, nullptr, rows, cols,
                              residual_scale, branch_scale, eps, order);
    if (s != TR_OK) return s;
    const bool pre = norms & TR_BLOCK_PRE, post = norms & TR_BLOCK_POST, layer = kind == TR_NORM_LAYER;
    if (!pre && dy) return fail(TR_ERR_INVALID_ARG, w, "dy needs TR_BLOCK_PRE");
    if ((!post && (dpost_w || dpost_b)) || (!pre && (dpre_w || dpre_b)) || (!layer && (dpost_b || dpre_b)) ||
        (!gate && dgate))
        return fail(TR_ERR_INVALID_ARG, w, "a gradient of a norm, bias or gate that is not there must be null");
    const bool sums = dpost_w || dpost_b || dgate || dpre_w || dpre_b;
    const size_t nc = static_cast<size_t>(cols) * 4, ng = gate ? nc * static_cast<size_t>(gate_rows) : 0;
    const size_t eb = element_bytes(dtype), n = static_cast<size_t>(rows) * cols * eb;
    const Range in[] = {{h, n, eb}, {branch, n, eb}, {dy, n, eb}, {dh, n, eb}, {post_w, nc, 4}, {post_b, nc, 4},
                        {pre_w, nc, 4}, {gate, ng, 4}};
    const Range out[] = {{dx, n, eb}, {dbranch, n, eb}, {dpost_w, nc, 4}, {dpost_b, nc, 4}, {dgate, ng, 4},
                         {dpre_w, nc, 4}, {dpre_b, nc, 4}, {workspace, sums ? workspace_bytes : 0, 16}};
    s = check_ranges(w, in, out);
    if (s != TR_OK) return s;
    if (rows == 0) {  // empty sums
        const Range zero[] = {{dpost_w, nc, 4}, {dpost_b, nc, 4}, {dgate, ng, 4}, {dpre_w, nc, 4}, {dpre_b, nc, 4}};
        for (const Range& r : zero) {
            if (!r.p) continue;
            const cudaError_t e = cudaMemsetAsync(const_cast<void*>(r.p), 0, r.bytes, stream);
            if (e != cudaSuccess) return cuda_status(e, w);
        }
        return TR_OK;
    }
    if (!dx || !dbranch) return fail(TR_ERR_INVALID_ARG, w, "dx and dbranch must not be null");
    if (pre && (!h || !dy)) return fail(TR_ERR_INVALID_ARG, w, "h and dy must not be null with TR_BLOCK_PRE");
    if (!pre && !dh) return fail(TR_ERR_INVALID_ARG, w, "dh must not be null without TR_BLOCK_PRE");
    if ((post || dgate) && !branch) return fail(TR_ERR_INVALID_ARG, w, "branch must not be null with TR_BLOCK_POST or dgate");
    if (sums && (!workspace || workspace_bytes < backward_bytes(kind, rows, cols)))
        return fail(TR_ERR_INVALID_ARG, w,
                    "the workspace is missing or smaller than tr_gated_residual_norm_backward_workspace_bytes");
    BlockBwArgs a{};
    a.h = h;
    a.a = branch;
    a.dy = dy;
    a.dh = dh;
    a.dx = dx;
    a.da = dbranch;
    a.post_w = post_w;
    a.post_b = post_b;
    a.gate = gate;
    a.pre_w = pre_w;
    a.dgate = dgate;
    a.dpost_w = dpost_w;
    a.dpost_b = dpost_b;
    a.dpre_w = dpre_w;
    a.dpre_b = dpre_b;
    a.rows = rows;
    a.groups = gate ? gate_rows : 1;
    a.group_rows = rows / a.groups;
    a.cols = static_cast<int>(cols);
    a.post = post ? 1 : 0;
    a.pre = pre ? 1 : 0;
    a.sums = sums ? 1 : 0;
    a.rs = residual_scale;
    a.bs = branch_scale;
    a.eps = eps;
    if (sums) {
        a.stats = static_cast<float*>(workspace);
        a.part = a.stats + stats_bytes(rows) / sizeof(float);
    }
    return guarded(w, [&] { return cuda_status(launch_block_backward(kind, dtype, a, stream), w); });
}

tr_status tr_global_norm_workspace_bytes(int64_t count, size_t* bytes) {
    static const char* w = "global norm workspace";
    if (!bytes) return fail(TR_ERR_INVALID_ARG, w, "bytes must not be null");
    if (count < 0 || count > (1LL << 31)) return fail(TR_ERR_INVALID_ARG, w, "count must be in [0, 2^31]");
    *bytes = norm_bytes(count);
    return TR_OK;
}

tr_status tr_global_norm(tr_total_kind kind, const void* const* tensors, const int64_t* numels, const int32_t* dtypes,
                         int64_t count, float* norm, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    static const char* w = "global norm";
    return guarded(w, [&] {
        int n = 0;
        const ListCall c{tensors, nullptr, numels, dtypes, count};
        const tr_status s = list_norm(w, kind, c, norm, workspace, workspace_bytes, &n, stream);
        if (s != TR_OK) return s;
        return cuda_status(launch_list_total(kind, static_cast<const double*>(workspace), n, norm, stream), w);
    });
}

tr_status tr_clip_by_norm(const void* const* tensors, void* const* outs, const int64_t* numels, const int32_t* dtypes,
                          int64_t count, const float* norm, float max_norm, float eps, cudaStream_t stream) {
    static const char* w = "clip by norm";
    return guarded(w, [&] {
        tr_status s = check_clip(w, max_norm, eps);
        if (s != TR_OK) return s;
        const ListCall c{tensors, outs ? outs : const_cast<void* const*>(tensors), numels, dtypes, count};
        s = check_list(w, c, norm, nullptr, 0);
        if (s == TR_OK && count > 0) s = check_written(w, c);
        if (s != TR_OK) return s;
        return scale_list(w, TR_TOTAL_L2, c, nullptr, 0, const_cast<float*>(norm), false, max_norm, eps, stream);
    });
}

tr_status tr_clip_global_norm(tr_total_kind kind, const void* const* tensors, void* const* outs,
                              const int64_t* numels, const int32_t* dtypes, int64_t count, float max_norm, float eps,
                              float* norm, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    static const char* w = "clip global norm";
    return guarded(w, [&] {
        tr_status s = check_clip(w, max_norm, eps);
        if (s != TR_OK) return s;
        const ListCall c{tensors, outs ? outs : const_cast<void* const*>(tensors), numels, dtypes, count};
        int n = 0;
        s = list_norm(w, kind, c, norm, workspace, workspace_bytes, &n, stream);
        if (s != TR_OK) return s;
        const double* part = static_cast<const double*>(workspace);
        if (n == 0) return cuda_status(launch_list_total(kind, part, 0, norm, stream), w);  // nothing to scale
        return scale_list(w, kind, c, part, n, norm, true, max_norm, eps, stream);
    });
}

}  // extern "C"
