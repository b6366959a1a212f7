// The on-chip gated residual norm on float rows.
#include "tr_block_fwd.cuh"

namespace tr {

cudaError_t launch_block_forward_f32(int kind, const BlockArgs& a, bool* done, cudaStream_t stream) {
    return kind == TR_NORM_LAYER ? block::fwd_kind<float, true>(a, done, stream) : block::fwd_kind<float, false>(a, done, stream);
}

}  // namespace tr
