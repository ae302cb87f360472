// block_vjp_f32.cu -- VJP instances of the norm pair around a block.
#include "block_launch.cuh"

namespace rmsn {
template <>
cudaError_t launch_block_vjp<float>(const BlockPlan &p, const BlockArgs &a, cudaStream_t s) {
    return launch_block_vjp_both<float>(p, a, s);
}
}  // namespace rmsn
