// Launch helpers of the block norms, the tensor lists, the embedding and the linear cross entropy.
#pragma once

#include <stddef.h>

#include <cuda_runtime.h>

namespace tr {

// CTAs of a kernel the current device holds at once (in clusters of `cluster`; asked once per
// kernel, size and device), its dynamic shared memory allowed; 0 when it cannot run.
int resident_ctas(const void* kernel, int threads, size_t smem, int cluster = 1);

// The current device's error word (null when it cannot be found).
unsigned* device_error_word();

// Launch so that this grid's start may overlap the previous kernel's end (the kernel
// waits in pdl_enter); TR_DISABLE_PDL=1 turns the overlap off.
bool dependent_launches();
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                             A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    if (dependent_launches()) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace tr
