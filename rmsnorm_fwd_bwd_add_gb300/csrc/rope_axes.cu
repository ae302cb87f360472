// rope_axes.cu -- rotary positions of several axes (time, height and width of image and
// video tokens): pair i of a token turns by the position on its own axis, t =
// positions[axis(i)][token] * inv_freq[i].
//
// Heads in 16-byte units go through the 8-bit append's kernel, whose warps compute a
// token's cosines together and copy heads ahead into shared memory (kv_cache8.cuh; without
// quantising): 16384 tokens of 32 + 8 heads of 128 57.3 us on rope_ex.cuh's kernel, 53.6 so.
// Smaller units stay on that one, with a choice of axis beside each pair.
#include "kv_append8.h"
#include "rope_ex.cuh"
#include "rope_host.h"

namespace rmsn {

namespace {

template <typename T> cudaError_t launch_small(const RopeArgs<true> &a, bool interleaved, int unit, int sm, cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (unit < 4) return interleaved ? launch_layout<T, 2, true, true>(a, sm, s) : launch_layout<T, 2, false, true>(a, sm, s);
    return interleaved ? launch_layout<T, 4, true, true>(a, sm, s) : launch_layout<T, 4, false, true>(a, sm, s);
}

template <typename T> cudaError_t launch_axes(const RopeArgs<true> &a, bool interleaved, int unit, int sm, cudaStream_t s) {
    const bool fits = interleaved ? append8_vectors_fit<T, true>(a.Dh, a.rot) : append8_vectors_fit<T, false>(a.Dh, a.rot);
    if (unit < 16 || !fits) return launch_small<T>(a, interleaved, unit, sm, s);
    AppendArgs b{};
    static_cast<RopeArgs<true> &>(b) = a;
    return interleaved ? launch_append8_vectors<T, true, RMSNORM_CACHE_SAME>(b, sm, s)
                       : launch_append8_vectors<T, false, RMSNORM_CACHE_SAME>(b, sm, s);
}

}  // namespace

cudaError_t launch_rope_axes(const RopeArgs<true> &a, bool interleaved, int unit, int dtype, int sm, cudaStream_t s) {
    return dtype == RMSNORM_F16    ? launch_axes<__half>(a, interleaved, unit, sm, s)
           : dtype == RMSNORM_BF16 ? launch_axes<__nv_bfloat16>(a, interleaved, unit, sm, s)
                                   : launch_axes<float>(a, interleaved, unit, sm, s);
}

}  // namespace rmsn
