// kv_append8_bf16.cu -- instances of the 8-bit append.
#include "kv_append8.h"

namespace rmsn {
template <>
cudaError_t launch_append8<__nv_bfloat16>(const AppendArgs &a, int format, bool interleaved, int unit, int sm, cudaStream_t s) {
    return launch_append8_any<__nv_bfloat16>(a, format, interleaved, unit, sm, s);
}
}  // namespace rmsn
