// block_fwd_bf16.cu -- forward instances of the norm pair around a block.
#include "block_launch.cuh"

namespace rmsn {
template <>
cudaError_t launch_block_fwd<__nv_bfloat16>(const BlockPlan &p, const BlockArgs &a, cudaStream_t s) {
    return launch_block<false, __nv_bfloat16>(p, a, s);
}
}  // namespace rmsn
