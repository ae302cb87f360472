// quant.cuh -- values in 8 bits: e4m3 and int8 codes of fp32 values, and the largest
// magnitude of a group.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"
#include "rmsnorm.h"

namespace rmsn {

// A cache's or output's format at compile time: its largest code.
template <int FMT> __host__ __device__ constexpr float top_code() { return FMT == RMSNORM_CACHE_I8 ? 127.f : 448.f; }

// The least magnitude a that a group's scale is made from: a / top and top / a are then
// normal numbers whatever the group holds.  (The norm's scale has its r as a factor beside
// them, and may be subnormal or 0.)
template <int FMT> __host__ __device__ constexpr float least_top() { return top_code<FMT>() * 0x1p-126f; }

// The largest magnitude among a group: NaN if any value is.
__device__ __forceinline__ float max_abs(float top, float a, float b) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(top), "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_abs(float top, float a) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(top), "f"(fabsf(a)));
    return r;
}
// Over all lanes of a warp, and over aligned runs of n lanes (a power of two).
__device__ __forceinline__ float warp_max(float top) {
    float r;
    asm volatile("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(top));
    return r;
}
__device__ __forceinline__ float run_max(float top, int n) {
    for (int off = 1; off < n; off *= 2) top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, off));
    return top;
}

// The magnitude that a group's scale is made from.
template <int FMT> __device__ __forceinline__ float scaled_top(float top) { return max_abs(least_top<FMT>(), top); }

// top_code / a for such an a, as the float nearest to it and the rest of it: an approximate
// reciprocal and one step of Newton's correction of the quotient, whose remainder gives the
// rest, on a brought down by a power of two so that neither a nor its reciprocal leaves the
// normal numbers.  NaN for a that is not finite.
template <int FMT> __device__ __forceinline__ float2 code_factor(float a) {
    constexpr float down = FMT == RMSNORM_CACHE_I8 ? 1.f / 64.f : 1.f / 256.f, n = top_code<FMT>() * down;
    const float x = a * down;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    const float q = n * r, hi = fmaf(fmaf(-q, x, n), r, q);
    return make_float2(hi, fmaf(-hi, x, n) * r);
}

// A value times such a factor, rounded once: the code of a 16-bit value is then that of the
// exact quotient, on the border of two codes too (with the factor's first part alone 10334
// e4m3 codes of 33 million bf16 values were not, with a division and a product in fp32 28654;
// int8 6884 and 12074).  It costs the append 2 % where heads are small (4096 tokens of 32 + 8
// heads of 100 30.7 -> 31.4 us) and nothing where memory bounds it (16384 of heads of 128).
__device__ __forceinline__ float in_codes(float x, float2 by) { return fmaf(x, by.x, x * by.y); }
__device__ __forceinline__ float2 in_codes(float2 x, float2 by) {
    return f2fma(x, make_float2(by.x, by.x), f2mul(x, make_float2(by.y, by.y)));
}

// Two values, times their scale's inverse already, as the codes' bytes (the first in
// the low byte), to nearest even.  e4m3: beyond 448 saturates, NaN stays NaN.
// int8: NaN is 0 (its scale is not a number).
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
    return r;
}
// One value at the nearest int8 code, in the low byte: beyond the range saturates.
__device__ __forceinline__ uint32_t i8_code(float a) {
    uint32_t r;
    asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(r) : "f"(a));
    return r & 0xffu;
}
template <int FMT> __device__ __forceinline__ uint32_t code_pair(float a, float b) {
    if constexpr (FMT == RMSNORM_CACHE_I8) return i8_code(a) | i8_code(b) << 8;
    else return e4m3_pair(a, b);
}
template <int FMT> __device__ __forceinline__ uint32_t code_quad(float a, float b, float c, float d) {
    return code_pair<FMT>(a, b) | code_pair<FMT>(c, d) << 16;
}

// Two codes (low and high byte of the low half) as floats.
template <int FMT> __device__ __forceinline__ float2 value_pair(uint32_t codes) {
    if constexpr (FMT == RMSNORM_CACHE_I8) {
        // 2^23 + 128 + code, whose last bits are the code's with its sign turned, less 2^23 + 128
        const uint32_t u = codes ^ 0x8080u;
        return f2add(make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7550)), __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7551))),
                     make_float2(-8388736.f, -8388736.f));
    } else {  // every e4m3 value is an fp16 one
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
        return Cvt<__half>::unpack2(h);
    }
}

}  // namespace rmsn
