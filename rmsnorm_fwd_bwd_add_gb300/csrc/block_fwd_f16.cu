// block_fwd_f16.cu -- forward instances of the norm pair around a block.
#include "block_launch.cuh"

namespace rmsn {
template <>
cudaError_t launch_block_fwd<__half>(const BlockPlan &p, const BlockArgs &a, cudaStream_t s) {
    return launch_block<false, __half>(p, a, s);
}
}  // namespace rmsn
