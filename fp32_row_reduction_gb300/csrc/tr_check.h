// Argument checks on the host that several entry points share.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <new>

#include <cuda_runtime.h>

#include "tr.h"
#include "tr_internal.h"

namespace tr {

inline tr_status fail(tr_status s, const char* where, const char* why) {
    set_last_error(where, why);
    return s;
}
// An error is also cleared from the runtime's last-error slot, which other entry points ask after their own launches.
inline tr_status cuda_status(cudaError_t e, const char* where) {
    if (e == cudaSuccess) return TR_OK;
    cudaGetLastError();
    return fail(TR_ERR_CUDA, where, cudaGetErrorString(e));
}

inline size_t element_bytes(int dtype) { return dtype == TR_F32 ? 4 : 2; }

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

}  // namespace tr
