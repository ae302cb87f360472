// block_fwd_f32.cu -- forward instances of the norm pair around a block.
#include "block_launch.cuh"

namespace rmsn {
template <>
cudaError_t launch_block_fwd<float>(const BlockPlan &p, const BlockArgs &a, cudaStream_t s) {
    return launch_block<false, float>(p, a, s);
}
}  // namespace rmsn
