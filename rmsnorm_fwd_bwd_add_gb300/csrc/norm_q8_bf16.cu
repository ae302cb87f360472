// norm_q8_bf16.cu -- instances of the 8-bit norm.
#include "norm_q8.cuh"

namespace rmsn {
template <>
cudaError_t launch_q8<__nv_bfloat16>(const Q8Plan &p, const Q8Args &a, cudaStream_t s) {
    return launch_q8_any<__nv_bfloat16>(p, a, s);
}
}  // namespace rmsn
