// block_vjp_f16.cu -- VJP instances of the norm pair around a block.
#include "block_launch.cuh"

namespace rmsn {
template <>
cudaError_t launch_block_vjp<__half>(const BlockPlan &p, const BlockArgs &a, cudaStream_t s) {
    return launch_block_vjp_both<__half>(p, a, s);
}
}  // namespace rmsn
