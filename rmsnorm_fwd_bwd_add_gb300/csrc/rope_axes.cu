// rope_axes.cu -- the rotary kernel for positions of several axes (time, height and
// width of image and video tokens): pair i of a token turns by the position on its
// own axis, t = positions[axis(i)][token] * inv_freq[i].
//
// The kernel is rope_ex.cu's: a lane computes the cosines and sines of its pairs once
// for all of the token's heads, so that the choice of axis costs a few selects a pair
// beside the loads and stores that bound it.
#include "rope_ex.cuh"
#include "rope_host.h"

namespace rmsn {

cudaError_t launch_rope_axes(const RopeArgs<true> &a, bool interleaved, int unit, int dtype, int sm, cudaStream_t s) {
    return launch_rope<true>(a, interleaved, unit, dtype, sm, s);
}

}  // namespace rmsn
