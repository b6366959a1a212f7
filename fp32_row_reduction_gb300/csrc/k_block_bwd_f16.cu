// The on-chip backward of the gated residual norm on __half rows.
#include "tr_block_bwd.cuh"

namespace tr {

cudaError_t launch_block_backward_f16(int kind, const BlockBwArgs& a, bool* done, cudaStream_t stream) {
    return kind == TR_NORM_LAYER ? block::bwd_kind<__half, true>(a, done, stream) : block::bwd_kind<__half, false>(a, done, stream);
}

}  // namespace tr
