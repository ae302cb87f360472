// units.cuh -- row elements in units of 16, 4 or 2 bytes: the widest that a
// call's addresses, strides and lengths allow.
#pragma once

#include "common.cuh"

namespace rmsn {

template <int UB> struct RawUnit;
template <> struct RawUnit<16> { using type = uint4; };
template <> struct RawUnit<4> { using type = uint32_t; };
template <> struct RawUnit<2> { using type = uint16_t; };

template <typename T, int UB> __host__ __device__ constexpr int unit_elems() { return UB / (int)sizeof(T); }

template <typename T, int UB>
__device__ __forceinline__ void unpack_unit(const typename RawUnit<UB>::type &v, float (&f)[unit_elems<T, UB>()]) {
    if constexpr (UB == 16) {
        unpack_vec<T>(v, f);
    } else {
        T x;
        memcpy(&x, &v, sizeof(T));
        f[0] = Cvt<T>::load1(&x);
    }
}

template <typename T, int UB>
__device__ __forceinline__ typename RawUnit<UB>::type pack_unit(const float (&f)[unit_elems<T, UB>()]) {
    if constexpr (UB == 16) {
        return pack_vec<T>(f);
    } else {
        T x;
        Cvt<T>::store1(&x, f[0]);
        typename RawUnit<UB>::type v;
        memcpy(&v, &x, sizeof(T));
        return v;
    }
}

}  // namespace rmsn
