// norm_q8.cuh -- kernels of the fused residual-add norm with an e4m3 output.
//
// With v_j = h_j w'_j and a = max |v_j| over a group, the group's scale is r a / 448 and
// its codes are e4m3(v_j 448 / a): the norm's own factor r is the same for the whole row
// and cancels in the codes, so that the row's sum of squares and the groups' maxima come
// from one pass.
#pragma once

#include "norm_q8.h"
#include "quant.cuh"
#include "units.cuh"

namespace rmsn {

constexpr int Q8_GENERIC_NT = 512;

// The scale of a group and the factor of its codes.
__device__ __forceinline__ float2 q8_scale(uint32_t top, float r) {
    // (integers: NaN and infinity stay)
    const float a = __uint_as_float(max(top, __float_as_uint(least_top<RMSNORM_CACHE_E4M3>())));
    return make_float2(r * a * (1.f / 448.f), 448.f / a);
}

// Any row length, stride and alignment: one element a thread, the row read twice (the
// second time from L2).  Groups go to a warp each.
template <typename T, bool RES>
__global__ void __launch_bounds__(Q8_GENERIC_NT) q8_generic_kernel(const Q8Args a) {
    constexpr int NW = Q8_GENERIC_NT / 32;
    __shared__ float s_sum[NW];
    __shared__ uint32_t s_top[NW];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T *w = static_cast<const T *>(a.w);
    griddep_wait();
    griddep_launch_dependents();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + row * a.ld_x;
        const T *res = RES ? static_cast<const T *>(a.res) + row * a.ld_res : nullptr;
        auto h_of = [&](int j) { return RES ? Cvt<T>::load1(x + j) + Cvt<T>::load1(res + j) : Cvt<T>::load1(x + j); };
        auto weight = [&](int j) { return a.weight_bias + Cvt<T>::load1(w + j); };
        // a sum of sums of 64, so that rounding grows with neither length alone
        float ss = 0.f;
        uint32_t top = 0;
        for (int j0 = threadIdx.x; j0 < a.D; j0 += 64 * Q8_GENERIC_NT) {
            float part = 0.f;
            for (int i = 0, j = j0; i < 64 && j < a.D; ++i, j += Q8_GENERIC_NT) {
                const float h = h_of(j);
                part = fmaf(h, h, part);
                if (!a.group) top = max(top, magnitude(h * weight(j)));
            }
            ss += part;
        }
        ss = group_sum<32>(ss);
        top = __reduce_max_sync(0xffffffffu, top);
        __syncthreads();  // the row before has been read
        if (lane == 0) {
            s_sum[warp] = ss;
            s_top[warp] = top;
        }
        __syncthreads();
        ss = group_sum<32>(lane < NW ? s_sum[lane] : 0.f);
        const float r = rsqrtf(ss * (1.0f / (float)a.D) + a.eps);
        uint8_t *out = static_cast<uint8_t *>(a.out) + row * a.ld_out;
        T *nres = RES ? static_cast<T *>(a.nres) + row * a.ld_nres : nullptr;
        auto write = [&](int j, float h, float by) {
            out[j] = (uint8_t)e4m3_pair(h * weight(j) * by, 0.f);
            if (RES) Cvt<T>::store1(nres + j, h);
        };
        if (!a.group) {
            top = __reduce_max_sync(0xffffffffu, lane < NW ? s_top[lane] : 0u);
            const float2 s = q8_scale(top, r);
            for (int j = threadIdx.x; j < a.D; j += Q8_GENERIC_NT) write(j, h_of(j), s.y);
            if (threadIdx.x == 0) a.scale[row] = s.x;
        } else {
            for (int g = warp; g < a.groups; g += NW) {
                float h[4];
                uint32_t t = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = g * a.group + 32 * i + lane;
                    const bool in = 32 * i < a.group && j < a.D;
                    h[i] = in ? h_of(j) : 0.f;
                    if (in) t = max(t, magnitude(h[i] * weight(j)));
                }
                const float2 s = q8_scale(__reduce_max_sync(0xffffffffu, t), r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = g * a.group + 32 * i + lane;
                    if (32 * i < a.group && j < a.D) write(j, h[i], s.y);
                }
                if (lane == 0) a.scale[row * a.groups + g] = s.x;
            }
        }
    }
}

}  // namespace rmsn
