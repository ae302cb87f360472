// block_vjp_bf16.cu -- VJP instances of the norm pair around a block.
#include "block_launch.cuh"

namespace rmsn {
template <>
cudaError_t launch_block_vjp<__nv_bfloat16>(const BlockPlan &p, const BlockArgs &a, cudaStream_t s) {
    return launch_block_vjp_both<__nv_bfloat16>(p, a, s);
}
}  // namespace rmsn
