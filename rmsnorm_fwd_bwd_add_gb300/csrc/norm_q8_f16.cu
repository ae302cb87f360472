// norm_q8_f16.cu -- instances of the 8-bit norm.
#include "norm_q8.cuh"

namespace rmsn {
template <>
cudaError_t launch_q8<__half>(const Q8Plan &p, const Q8Args &a, cudaStream_t s) {
    return launch_q8_any<__half>(p, a, s);
}
}  // namespace rmsn
