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

// Codes of VE elements as one word.
template <int VE> struct CodeWord;
template <> struct CodeWord<8> { using type = uint2; };
template <> struct CodeWord<4> { using type = uint32_t; };
template <> struct CodeWord<2> { using type = uint16_t; };

template <int FMT, int VE> __device__ __forceinline__ typename CodeWord<VE>::type code_word(const float (&f)[VE], float by) {
    if constexpr (VE == 8) {
        return make_uint2(code_quad<FMT>(f[0] * by, f[1] * by, f[2] * by, f[3] * by),
                          code_quad<FMT>(f[4] * by, f[5] * by, f[6] * by, f[7] * by));
    } else if constexpr (VE == 4) {
        return code_quad<FMT>(f[0] * by, f[1] * by, f[2] * by, f[3] * by);
    } else {
        return (uint16_t)code_pair<FMT>(f[0] * by, f[1] * by);
    }
}

template <typename T, int VB, int VE> __device__ __forceinline__ void unpack_raw(const typename RawUnit<VB>::type &v, float (&f)[VE]) {
    if constexpr (VB == 16) {
        unpack_vec<T>(v, f);
    } else {
        const float2 p = Cvt<T>::unpack2(v);
        f[0] = p.x;
        f[1] = p.y;
    }
}
template <typename T, int VB, int VE> __device__ __forceinline__ typename RawUnit<VB>::type pack_raw(const float (&f)[VE]) {
    if constexpr (VB == 16) return pack_vec<T>(f);
    else return Cvt<T>::pack2(f[0], f[1]);
}

// Units of a head a lane holds at a time, over all heads in flight.
constexpr int C8_UNITS_IN_FLIGHT = 4;

// CTAs an SM holds: long heads need twice the registers for their cosines and sines.
template <int VE, int UPL> __host__ __device__ constexpr int append8_ctas() { return VE * UPL > 8 ? 1 : 2; }

// A warp takes a token (or one of a token's `wpt` parts, from token `whole` on), 32 / cw
// heads at a time: cw lanes a head, UPL units of two vectors each a lane (rope_ex.cuh's
// units), so that a head's largest value is a few shuffles away.  The cosines and sines
// of a lane's pairs are computed once for all of its heads.
template <typename T, int VB, bool INTERLEAVED, int FMT, int UPL>
__global__ void __launch_bounds__(C8_NT, (append8_ctas<VB / (int)sizeof(T), UPL>())) append8_kernel(const __grid_constant__ AppendArgs a, int64_t whole, int wpt, int cw) {
    using V = typename RawUnit<VB>::type;
    constexpr int VE = VB / (int)sizeof(T), HB = C8_UNITS_IN_FLIGHT / UPL;
    constexpr bool PAIRED = INTERLEAVED;  // VE > 1
    using Codes = typename CodeWord<VE>::type;
    __shared__ float2 s_turns[RX_MAX_DH / 2];
    __shared__ uint8_t s_axis[RX_MAX_DH / 2];
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < half; i += C8_NT) {
        s_turns[i] = a.turns[i];
        s_axis[i] = a.axes.of[i];
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();

    const int lane = threadIdx.x & 31, hpi = 32 / cw, hs = lane / cw, lu = lane - hs * cw;
    const HeadMap<VE, PAIRED, INTERLEAVED> map(a.Dh, a.rot), v_map(a.Dh, 0);
    const bool q_moves = a.q_out.p != a.q.p;  // in place: nothing to copy
    const int n_qk = a.Hq + a.Hkv, n_all = n_qk + a.Hkv;
    // unit i of this lane: first elements of its two vectors in a head of q or k, and of v
    int ia[UPL], ib[UPL], va[UPL], vb[UPL];
    uint32_t in = 0, two = 0, turns = 0, v_in = 0, v_two = 0;  // a bit a unit
#pragma unroll
    for (int i = 0; i < UPL; ++i) {
        const int l = lu + i * cw;
        bool w;
        map.at(l, ia[i], ib[i], w);
        if (l < map.lanes) in |= 1u << i, two |= (uint32_t)w << i;
        if (l < map.rot_units) turns |= 1u << i;
        v_map.at(l, va[i], vb[i], w);
        if (l < v_map.lanes) v_in |= 1u << i, v_two |= (uint32_t)w << i;
    }
    const int64_t n_items = whole + (a.T - whole) * wpt, n_warps = (int64_t)gridDim.x * (C8_NT / 32);
    const int wshift = 31 - __clz(wpt);  // wpt is a power of two
    int64_t w = ((int64_t)blockIdx.x * C8_NT + threadIdx.x) >> 5;
    int64_t p_next[RX_MAX_AXES] = {}, slot_next = 0;  // of the item ahead
    auto token_of = [&](int64_t item) { return item < whole ? item : whole + ((item - whole) >> wshift); };
    auto look_ahead = [&](int64_t item) {
        if (item < n_items) {
            const int64_t t = token_of(item);
            slot_next = a.slots[t];
#pragma unroll
            for (int x = 0; x < RX_MAX_AXES; ++x)
                if (x < a.axes.n) p_next[x] = a.positions[x * a.T + t];
        }
    };
    look_ahead(w);
    for (; w < n_items; w += n_warps) {
        const int64_t t = token_of(w), slot = slot_next;
        float2 pos[RX_MAX_AXES];
        bool pos_ok = true;
#pragma unroll
        for (int x = 0; x < RX_MAX_AXES; ++x) {
            pos[x] = split_position(p_next[x]);
            pos_ok = pos_ok && p_next[x] >= 0;
        }
        const int parts = w < whole ? 1 : wpt, part = w < whole ? 0 : (int)((w - whole) & (wpt - 1));
        look_ahead(w + n_warps);
        const bool slot_ok = slot < a.num_slots;
        if ((!pos_ok || !slot_ok) && lane == 0 && part == 0) atomicOr(a.status, BAD_INDEX);
        if (!pos_ok) continue;
        const int heads = slot_ok && slot >= 0 ? n_all : a.Hq;
        auto place = [&](const Heads &x, int64_t row, int es, int before) {
            return (unsigned char *)x.p + (row * x.st * es - (int64_t)before * x.head_bytes);
        };
        const unsigned char *q = place(a.q, t, sizeof(T), 0), *k = place(a.k, t, sizeof(T), a.Hq), *v = place(a.v, t, sizeof(T), n_qk);
        unsigned char *qo = place(a.q_out, t, sizeof(T), 0), *ko = place(a.k_out, slot, 1, a.Hq), *vo = place(a.v_out, slot, 1, n_qk);
        // of a head's pairs; quantised values take sines to fp32's precision: the SFU's
        // (2^-21) would move values across the codes' borders
        float cs[UPL][VE], sn[UPL][VE];
#pragma unroll
        for (int i = 0; i < UPL; ++i)
            if (turns >> i & 1) {
#pragma unroll
                for (int m = 0; m < VE; ++m) {
                    const int pair = !PAIRED ? ia[i] + m : m < VE / 2 ? ia[i] / 2 + m : min(ib[i] / 2 + m - VE / 2, half - 1);
                    const int axis = s_axis[pair];
                    float2 p = pos[0];
#pragma unroll
                    for (int x = 1; x < RX_MAX_AXES; ++x) p = axis == x ? pos[x] : p;
                    const float2 c = cos_sin<true>(p, s_turns[pair]);
                    cs[i][m] = c.x * a.scale;
                    sn[i][m] = c.y * a.scale;
                }
            }
        const int step = parts * hpi;
        for (int hb = part * hpi; hb < heads; hb += HB * step) {
            V xa[HB][UPL], xb[HB][UPL];
#pragma unroll
            for (int j = 0; j < HB; ++j) {
                const int h = hb + j * step + hs;
                if (hs >= hpi || h >= heads) continue;
                const bool is_v = h >= n_qk;
                const unsigned char *base = h < a.Hq ? q : is_v ? v : k;
                const uint32_t sh = h < a.Hq ? a.q.head_bytes : is_v ? a.v.head_bytes : a.k.head_bytes;
                const T *src = reinterpret_cast<const T *>(base + (uint64_t)(uint32_t)h * sh);
                const uint32_t wanted = is_v ? v_in : h < a.Hq && !q_moves ? turns : in, both = is_v ? v_two : two;
#pragma unroll
                for (int i = 0; i < UPL; ++i)
                    if (wanted >> i & 1) {
                        xa[j][i] = *reinterpret_cast<const V *>(src + (is_v ? va[i] : ia[i]));
                        if (both >> i & 1) xb[j][i] = *reinterpret_cast<const V *>(src + (is_v ? vb[i] : ib[i]));
                    }
            }
#pragma unroll
            for (int j = 0; j < HB; ++j) {
                const int first = hb + j * step;  // the same in the whole warp
                if (first >= heads) break;
                const int h = first + hs;
                const bool mine = hs < hpi && h < heads, is_q = h < a.Hq, is_v = h >= n_qk;
                const uint32_t wanted = !mine ? 0u : is_v ? v_in : is_q && !q_moves ? turns : in, both = is_v ? v_two : two;
                float fa[UPL][VE], fb[UPL][VE];
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < UPL; ++i)
                    if (wanted >> i & 1) {
                        unpack_raw<T, VB>(xa[j][i], fa[i]);
                        if (both >> i & 1) unpack_raw<T, VB>(xb[j][i], fb[i]);
                        else
#pragma unroll
                            for (int e = 0; e < VE; ++e) fb[i][e] = 0.f;
                        if (!is_v && (turns >> i & 1)) {
                            if constexpr (PAIRED) {
                                auto pairs = [&](float (&f)[VE], int from) {
#pragma unroll
                                    for (int m = 0; m < VE / 2; ++m) {
                                        const float x = f[2 * m], y = f[2 * m + 1], c = cs[i][from + m], s = sn[i][from + m];
                                        f[2 * m] = fmaf(-y, s, x * c);
                                        f[2 * m + 1] = fmaf(x, s, y * c);
                                    }
                                };
                                pairs(fa[i], 0);
                                pairs(fb[i], VE / 2);
                            } else {
#pragma unroll
                                for (int m = 0; m < VE; ++m) {
                                    const float x = fa[i][m], y = fb[i][m], c = cs[i][m], s = sn[i][m];
                                    fa[i][m] = fmaf(-y, s, x * c);
                                    fb[i][m] = fmaf(x, s, y * c);
                                }
                            }
                        }
                        if (is_q) {
                            T *dst = reinterpret_cast<T *>(qo + (uint64_t)(uint32_t)h * a.q_out.head_bytes);
                            *reinterpret_cast<V *>(dst + ia[i]) = pack_raw<T, VB>(fa[i]);
                            if (both >> i & 1) *reinterpret_cast<V *>(dst + ib[i]) = pack_raw<T, VB>(fb[i]);
                        } else {
#pragma unroll
                            for (int e = 0; e < VE; ++e) top = max_abs(top, fa[i][e], fb[i][e]);
                        }
                    }
                if (first + hpi <= a.Hq) continue;  // heads of q alone
                // the largest of the head's cw lanes (counting some twice does no harm)
                for (int off = 1; off < cw; off *= 2) {
                    const int at = lu + off;
                    top = max_abs(top, __shfl_sync(0xffffffffu, top, hs < hpi ? lane - lu + (at < cw ? at : at - cw) : lane));
                }
                if (!mine || is_q) continue;
                const float most = scaled_top<FMT>(top);
                const float by = code_factor<FMT>(most);
                unsigned char *dst = (is_v ? vo : ko) + (uint64_t)(uint32_t)h * (is_v ? a.v_out.head_bytes : a.k_out.head_bytes);
#pragma unroll
                for (int i = 0; i < UPL; ++i)
                    if (wanted >> i & 1) {
                        *reinterpret_cast<Codes *>(dst + (is_v ? va[i] : ia[i])) = code_word<FMT>(fa[i], by);
                        if (both >> i & 1) *reinterpret_cast<Codes *>(dst + (is_v ? vb[i] : ib[i])) = code_word<FMT>(fb[i], by);
                    }
                if (lu == 0) {
                    const float scale = most * (1.f / top_code<FMT>());
                    if (is_v) a.v_scale.p[slot * a.v_scale.st + (h - n_qk) * a.v_scale.sh] = scale;
                    else a.k_scale.p[slot * a.k_scale.st + (h - a.Hq) * a.k_scale.sh] = scale;
                }
            }
        }
    }
}

// Any stride, alignment and head: a warp a head of a token, a lane its elements 32
// apart, which a head of k or v computes twice: for its largest and for its codes.
template <typename T, int FMT, bool INTERLEAVED>
__global__ void __launch_bounds__(C8_NT) append8_generic_kernel(const __grid_constant__ AppendArgs a) {
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
                const float2 cs = cos_sin<true>(p, a.turns[m]);
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
        float top = 0.f;
        each([&](int, float u, int, float w) { top = max_abs(top, u, w); });
        const float most = scaled_top<FMT>(warp_max(top));
        const float by = code_factor<FMT>(most);
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

// C codes as one load, and C elements as 16-byte stores or one of less.
template <int C> struct CodeLoad;
template <> struct CodeLoad<16> { using type = uint4; };
template <> struct CodeLoad<8> { using type = uint2; };
template <> struct CodeLoad<4> { using type = uint32_t; };
template <> struct CodeLoad<2> { using type = uint16_t; };
template <> struct CodeLoad<1> { using type = uint8_t; };

template <typename T, int FMT, int C>
__device__ __forceinline__ void write_values(T *out, const typename CodeLoad<C>::type &codes, float by) {
    uint32_t w[(C + 3) / 4] = {};
    memcpy(w, &codes, sizeof(codes));
    float f[C < 2 ? 2 : C];
#pragma unroll
    for (int i = 0; i < (C + 1) / 2; ++i) {
        const float2 v = value_pair<FMT>(w[i / 2] >> (16 * (i % 2)) & 0xffffu);
        f[2 * i] = v.x * by;
        f[2 * i + 1] = v.y * by;
    }
    constexpr int E = vec_elems<T>();
    if constexpr (C >= E) {
#pragma unroll
        for (int i = 0; i < C / E; ++i) {
            float g[E];
#pragma unroll
            for (int e = 0; e < E; ++e) g[e] = f[i * E + e];
            reinterpret_cast<uint4 *>(out)[i] = pack_vec<T>(g);
        }
    } else if constexpr (C == 1) {
        Cvt<T>::store1(out, f[0]);
    } else if constexpr (sizeof(T) == 4) {  // C == 2
        *reinterpret_cast<float2 *>(out) = make_float2(f[0], f[1]);
    } else if constexpr (C == 4) {
        *reinterpret_cast<uint2 *>(out) = make_uint2(Cvt<T>::pack2(f[0], f[1]), Cvt<T>::pack2(f[2], f[3]));
    } else {
        *reinterpret_cast<uint32_t *>(out) = Cvt<T>::pack2(f[0], f[1]);
    }
}

constexpr int R8_CTAS_PER_SM = 4;
constexpr int R8_IN_FLIGHT = 4;

// A warp takes a token's k and v, or one of a token's `wpt` parts: a unit of C codes a
// lane at a time, R8_IN_FLIGHT of them loaded ahead of their stores.
template <typename T, int FMT, int C>
__global__ void __launch_bounds__(C8_NT, R8_CTAS_PER_SM) read8_kernel(const __grid_constant__ ReadArgs a, int wpt) {
    using L = typename CodeLoad<C>::type;
    const int lane = threadIdx.x & 31, U = a.Dh / C, heads = 2 * a.Hkv;
    const int step = 32 * wpt, step_h = step / U, step_u = step - step_h * U;
    const int64_t n_items = a.T * wpt, n_warps = (int64_t)gridDim.x * (C8_NT / 32);
    const int shift = 31 - __clz(wpt);  // wpt is a power of two
    griddep_wait();
    griddep_launch_dependents();
    int64_t w = ((int64_t)blockIdx.x * C8_NT + threadIdx.x) >> 5, next = w < n_items ? a.slots[w >> shift] : 0;
    for (; w < n_items; w += n_warps) {
        const int64_t t = w >> shift, slot = next;
        const int part = (int)(w & (wpt - 1));
        if (w + n_warps < n_items) next = a.slots[(w + n_warps) >> shift];
        const bool there = slot >= 0 && slot < a.num_slots;
        if (slot >= a.num_slots && lane == 0 && part == 0) atomicOr(a.status, BAD_INDEX);
        // where heads 0 of k and v would be, counted through the list of both
        const uint8_t *k = static_cast<const uint8_t *>(a.k.p) + slot * a.k.st;
        const uint8_t *v = static_cast<const uint8_t *>(a.v.p) + slot * a.v.st;
        const float *ks = a.k_scale.p + slot * a.k_scale.st, *vs = a.v_scale.p + slot * a.v_scale.st;
        T *ko = static_cast<T *>(const_cast<void *>(a.k_out.p)) + t * a.k_out.st;
        T *vo = static_cast<T *>(const_cast<void *>(a.v_out.p)) + t * a.v_out.st;
        int h = (32 * part + lane) / U, u = 32 * part + lane - h * U;
        while (h < heads) {
            L codes[R8_IN_FLIGHT];
            float by[R8_IN_FLIGHT];
            T *out[R8_IN_FLIGHT];
#pragma unroll
            for (int i = 0; i < R8_IN_FLIGHT; ++i) {
                codes[i] = L{};
                by[i] = 0.f;
                out[i] = nullptr;
                if (h < heads) {
                    const bool is_v = h >= a.Hkv;
                    const int64_t hk = is_v ? h - a.Hkv : h;
                    out[i] = (is_v ? vo + hk * a.v_out.sh : ko + hk * a.k_out.sh) + u * C;
                    if (there) {
                        codes[i] = *reinterpret_cast<const L *>((is_v ? v + hk * a.v.sh : k + hk * a.k.sh) + u * C);
                        by[i] = is_v ? vs[hk * a.v_scale.sh] : ks[hk * a.k_scale.sh];
                    }
                }
                h += step_h;
                u += step_u;
                if (u >= U) {
                    u -= U;
                    ++h;
                }
            }
#pragma unroll
            for (int i = 0; i < R8_IN_FLIGHT; ++i)
                if (out[i]) write_values<T, FMT, C>(out[i], codes[i], by[i]);
        }
    }
}

}  // namespace rmsn
