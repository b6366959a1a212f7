// The on-chip gated residual norm on __half rows.
#include "tr_block_fwd.cuh"

namespace tr {

cudaError_t launch_block_forward_f16(int kind, const BlockArgs& a, bool* done, cudaStream_t stream) {
    return kind == TR_NORM_LAYER ? block::fwd_kind<__half, true>(a, done, stream) : block::fwd_kind<__half, false>(a, done, stream);
}

}  // namespace tr
