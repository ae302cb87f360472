// kv_append8.h -- the 8-bit append's launchers of one input type each
// (kv_append8_<type>.cu; the kernels are in kv_cache8.cuh).
#pragma once

#include "kv_cache8.cuh"

namespace rmsn {

// unit: bytes that divide every address, stride and length of q, k, v and q_out, and in
// elements those of the caches: 16 or 4, or less.
template <typename T> cudaError_t launch_append8(const AppendArgs &a, int format, bool interleaved, int unit, int sm, cudaStream_t s);

template <typename T, int VB, bool INTERLEAVED, int FMT, int UPL>
cudaError_t launch_append8_units(const AppendArgs &a, int lanes, int sm, cudaStream_t s) {
    if (lanes < 1 || lanes > 32 * UPL) return cudaErrorInvalidConfiguration;  // a head's lanes are a warp's
    static std::atomic<uint64_t> smem_mask{0};
    auto kern = append8_kernel<T, VB, INTERLEAVED, FMT, UPL>;
    const cudaError_t e = allow_max_dynamic_smem((const void *)kern, smem_mask);
    if (e != cudaSuccess) return e;
    const Append8Plan p = make_append8_plan(a.T, (lanes + UPL - 1) / UPL, a.Hq, a.Hkv, a.slots ? 2 : 1, a.rot / 2, UPL,
                                            sm * C8_CTAS_PER_SM, C8_NT / 32);
    const size_t smem = (size_t)(C8_NT / 32) * (append8_ring<VB, UPL, FMT>() * append8_step_bytes<VB, UPL>(a.Dh * (int)sizeof(T), p.cw) +
                                                2 * append8_plane(a.rot) * sizeof(float));
    return launch_pdl(kern, dim3(p.grid), dim3(C8_NT), smem, s, a, p.whole, p.wpt, p.cw);
}

// Lanes of a head in units of VE elements.
template <int VE, bool INTERLEAVED> int head_lanes(int Dh, int rot) {
    return HeadMap<VE, (INTERLEAVED && VE > 1), INTERLEAVED>(Dh, rot).lanes;
}

// Whether a warp's lanes hold a head in 16-byte units.  An odd number of vectors in both
// its parts takes a lane more than their sum: one of 1024 elements then does not fit.
template <typename T, bool INTERLEAVED> bool append8_vectors_fit(int Dh, int rot) {
    constexpr int E = 16 / (int)sizeof(T);
    return head_lanes<E, INTERLEAVED>(Dh, rot) <= 32 * (16 / E);
}

// Heads in 16-byte units, 16 elements a lane while a head's lanes are a warp's.
template <typename T, bool INTERLEAVED, int FMT>
cudaError_t launch_append8_vectors(const AppendArgs &a, int sm, cudaStream_t s) {
    constexpr int E = 16 / (int)sizeof(T);
    const int lanes = head_lanes<E, INTERLEAVED>(a.Dh, a.rot);
    if (lanes <= 32 * (8 / E)) return launch_append8_units<T, 16, INTERLEAVED, FMT, 8 / E>(a, lanes, sm, s);
    return launch_append8_units<T, 16, INTERLEAVED, FMT, 16 / E>(a, lanes, sm, s);
}

// Smaller units: fewer lanes a head leave each step less work beside its elements (4096
// tokens of 32 + 8 heads of 100 in 4-byte units: 53 us with 4 elements a lane, 36 with 8, 31
// with 16), until they spill (of 126 in single elements 60 us with 4, 46 with 8, 62 with 16,
// which heads of over 256 take).  Heads of over 512 go to the kernel of a warp a head.
template <typename T, bool INTERLEAVED, int FMT>
cudaError_t launch_append8_layout(const AppendArgs &a, int unit, int sm, cudaStream_t s) {
    if (unit == 16 && append8_vectors_fit<T, INTERLEAVED>(a.Dh, a.rot)) return launch_append8_vectors<T, INTERLEAVED, FMT>(a, sm, s);
    if constexpr (sizeof(T) == 2)
        if (unit >= 4) {
            const int lanes = head_lanes<2, INTERLEAVED>(a.Dh, a.rot);
            if (lanes <= 128) return launch_append8_units<T, 4, INTERLEAVED, FMT, 4>(a, lanes, sm, s);
        }
    const int lanes = head_lanes<1, INTERLEAVED>(a.Dh, a.rot);
    if (lanes <= 128) return launch_append8_units<T, (int)sizeof(T), INTERLEAVED, FMT, 4>(a, lanes, sm, s);
    if (lanes <= 256) return launch_append8_units<T, (int)sizeof(T), INTERLEAVED, FMT, 8>(a, lanes, sm, s);
    const int64_t warps = a.T * (a.Hq + 2 * (int64_t)a.Hkv);
    const dim3 grid((unsigned)std::min<int64_t>((warps + C8_NT / 32 - 1) / (C8_NT / 32), 8 * (int64_t)sm));
    return launch_pdl(append8_generic_kernel<T, FMT, INTERLEAVED>, grid, dim3(C8_NT), 0, s, a);
}

template <typename T>
cudaError_t launch_append8_any(const AppendArgs &a, int format, bool interleaved, int unit, int sm, cudaStream_t s) {
    if (format == RMSNORM_CACHE_I8)
        return interleaved ? launch_append8_layout<T, true, RMSNORM_CACHE_I8>(a, unit, sm, s)
                           : launch_append8_layout<T, false, RMSNORM_CACHE_I8>(a, unit, sm, s);
    return interleaved ? launch_append8_layout<T, true, RMSNORM_CACHE_E4M3>(a, unit, sm, s)
                       : launch_append8_layout<T, false, RMSNORM_CACHE_E4M3>(a, unit, sm, s);
}

}  // namespace rmsn
