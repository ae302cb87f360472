// kv_cache8.cuh -- kernels of the 8-bit cache: the append that rotates, quantises and
// writes a step's tokens, and the read that brings them back.
#pragma once

#include "quant.cuh"
#include "rope_ex.cuh"

namespace rmsn {

constexpr int C8_NT = 256;

// [num_slots, Hkv] scales: strides in elements.
struct Scales {
    float *p;
    int64_t st, sh;
};

struct AppendArgs : RopeArgs<true> {
    Scales k_scale, v_scale;
};

// Any stride, alignment and head: a warp a head of a token, a lane its elements 32
// apart, which a head of k or v computes twice: for its largest and for its codes.
template <typename T, int FMT, bool INTERLEAVED>
__global__ void __launch_bounds__(C8_NT) append8_generic_kernel(const __grid_constant__ AppendArgs a) {
    constexpr bool PRECISE = sizeof(T) == 4;
    const int lane = threadIdx.x & 31, half = a.rot / 2;
    const int heads = a.Hq + 2 * a.Hkv;
    const int64_t n_items = a.T * heads, n_warps = (int64_t)gridDim.x * (C8_NT / 32);
    griddep_wait();
    griddep_launch_dependents();
    for (int64_t item = ((int64_t)blockIdx.x * C8_NT + threadIdx.x) >> 5; item < n_items; item += n_warps) {
        const int64_t t = item / heads, slot = a.slots[t];
        const int h = (int)(item - t * heads);
        float2 pos[RX_MAX_AXES];
        bool pos_ok = true;
        for (int x = 0; x < RX_MAX_AXES; ++x) {
            const int64_t p = x < a.axes.n ? a.positions[x * a.T + t] : 0;
            pos[x] = split_position(p);
            pos_ok = pos_ok && p >= 0;
        }
        const bool slot_ok = slot < a.num_slots;
        if ((!pos_ok || !slot_ok) && lane == 0 && h == 0) atomicOr(a.status, BAD_INDEX);
        if (!pos_ok) continue;
        const int what = h < a.Hq ? 0 : h < a.Hq + a.Hkv ? 1 : 2, hk = h - (what == 0 ? 0 : what == 1 ? a.Hq : a.Hq + a.Hkv);
        if (what && (!slot_ok || slot < 0)) continue;
        const Heads &src = what == 0 ? a.q : what == 1 ? a.k : a.v;
        const T *x = static_cast<const T *>(src.p) + t * src.st + hk * src.sh;
        const int rot = what == 2 ? 0 : a.rot;  // v is copied
        // f(i, x_i, j, x_j) for each pair, f(i, x_i, -1, 0) for each element behind them
        auto each = [&](auto f) {
            for (int m = lane; m < rot / 2; m += 32) {
                const int i = INTERLEAVED ? 2 * m : m, j = INTERLEAVED ? i + 1 : m + half;
                float2 p = pos[0];
                for (int n = 1; n < RX_MAX_AXES; ++n) p = a.axes.of[m] == n ? pos[n] : p;
                const float2 cs = cos_sin<PRECISE>(p, a.turns[m]);
                const float c = cs.x * a.scale, s = cs.y * a.scale;
                const float u = Cvt<T>::load1(x + i), w = Cvt<T>::load1(x + j);
                f(i, fmaf(-w, s, u * c), j, fmaf(u, s, w * c));
            }
            for (int i = rot + lane; i < a.Dh; i += 32) f(i, Cvt<T>::load1(x + i), -1, 0.f);
        };
        if (what == 0) {
            T *o = static_cast<T *>(const_cast<void *>(a.q_out.p)) + t * a.q_out.st + hk * a.q_out.sh;
            each([&](int i, float u, int j, float w) {
                Cvt<T>::store1(o + i, u);
                if (j >= 0) Cvt<T>::store1(o + j, w);
            });
            continue;
        }
        uint32_t top = 0;
        each([&](int, float u, int, float w) { top = max(top, max(magnitude(u), magnitude(w))); });
        top = __reduce_max_sync(0xffffffffu, top);
        const float most = __uint_as_float(max(top, __float_as_uint(least_top<FMT>())));
        const float by = top_code<FMT>() / most;
        const Heads &dst = what == 1 ? a.k_out : a.v_out;
        uint8_t *o = static_cast<uint8_t *>(const_cast<void *>(dst.p)) + slot * dst.st + hk * dst.sh;
        each([&](int i, float u, int j, float w) {
            const uint32_t c = code_pair<FMT>(u * by, w * by);
            o[i] = (uint8_t)c;
            if (j >= 0) o[j] = (uint8_t)(c >> 8);
        });
        const Scales &sc = what == 1 ? a.k_scale : a.v_scale;
        if (lane == 0) sc.p[slot * sc.st + hk * sc.sh] = most * (1.f / top_code<FMT>());
    }
}

struct ReadArgs {
    Heads k, v, k_out, v_out;  // caches in codes, outputs in elements
    Scales k_scale, v_scale;
    const int64_t *slots;
    int64_t T, num_slots;
    int Hkv, Dh;
    unsigned int *status;
};

// Any stride, alignment and head: a warp a head of k or v of a token.
template <typename T, int FMT>
__global__ void __launch_bounds__(C8_NT) read8_generic_kernel(const __grid_constant__ ReadArgs a) {
    const int lane = threadIdx.x & 31, heads = 2 * a.Hkv;
    const int64_t n_items = a.T * heads, n_warps = (int64_t)gridDim.x * (C8_NT / 32);
    griddep_wait();
    griddep_launch_dependents();
    for (int64_t item = ((int64_t)blockIdx.x * C8_NT + threadIdx.x) >> 5; item < n_items; item += n_warps) {
        const int64_t t = item / heads, slot = a.slots[t];
        const int h = (int)(item - t * heads);
        const bool is_v = h >= a.Hkv, there = slot >= 0 && slot < a.num_slots;
        const int hk = is_v ? h - a.Hkv : h;
        if (slot >= a.num_slots && lane == 0 && h == 0) atomicOr(a.status, BAD_INDEX);
        const Heads &src = is_v ? a.v : a.k, &dst = is_v ? a.v_out : a.k_out;
        const Scales &sc = is_v ? a.v_scale : a.k_scale;
        const uint8_t *c = static_cast<const uint8_t *>(src.p) + slot * src.st + hk * src.sh;
        T *o = static_cast<T *>(const_cast<void *>(dst.p)) + t * dst.st + hk * dst.sh;
        const float by = there ? sc.p[slot * sc.st + hk * sc.sh] : 0.f;
        for (int i = lane; i < a.Dh; i += 32)
            Cvt<T>::store1(o + i, there ? value_pair<FMT>(c[i]).x * by : 0.f);
    }
}

}  // namespace rmsn
