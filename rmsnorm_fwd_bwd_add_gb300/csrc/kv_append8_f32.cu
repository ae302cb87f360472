// kv_append8_f32.cu -- instances of the 8-bit append.
#include "kv_append8.h"

namespace rmsn {
template <>
cudaError_t launch_append8<float>(const AppendArgs &a, int format, bool interleaved, int unit, int sm, cudaStream_t s) {
    return launch_append8_any<float>(a, format, interleaved, unit, sm, s);
}
}  // namespace rmsn
