// rope_ex.cuh -- the rotary kernel of rope_ex.cu and rope_axes.cu.
#pragma once

#include "rmsnorm.h"

#include "common.cuh"
#include "heads.h"
#include "launch_util.h"
#include "rope_plan.h"
#include "units.cuh"

namespace rmsn {

constexpr int RX_NT = 256;
constexpr int RX_CTAS_PER_SM = 2;
constexpr int RX_MAX_DH = 1024;
constexpr unsigned int BAD_INDEX = RMSNORM_DEVSTATUS_BAD_INDEX;

struct RopeExArgs {
    float2 turns[RX_MAX_DH / 2];  // (hi, lo) of inv_freq / 2 pi
    Heads q, k, v, q_out, k_out, v_out;
    const int64_t *positions, *slots;  // slots: null without a cache
    int64_t T, S, num_slots;
    int Hq, Hkv, Dh, rot;
    float scale, sign;
    unsigned int *status;
};

// Positions of several axes (time, height, width): [axes, T], and the axis that each
// pair turns by.
constexpr int RX_MAX_AXES = RMSNORM_ROPE_MAX_AXES;
struct RopeAxes {
    int n;
    uint8_t of[RX_MAX_DH / 2];
};
template <bool AXES> struct RopeArgs : RopeExArgs {};
template <> struct RopeArgs<true> : RopeExArgs {
    RopeAxes axes;
};

// A position as the float nearest to it and the rest.
__device__ __forceinline__ float2 split_position(int64_t p) {
    const float ph = (float)p;
    return make_float2(ph, (float)(p - (int64_t)ph));
}

// (cos, sin) of a position times a frequency in turns.  PRECISE (fp32 results, and values
// that become codes): what the reduced angle loses in its last addition, 2^-26 turns, three
// times the error of the sines themselves, is added to first order (the fp32 rotation's
// error against 64 bits 4.9e-8 without it, 4.1e-8 with it and with 64-bit angles; of 17
// million e4m3 codes of k 45 and 24 differ from 64-bit values', many times that with the
// SFU's sines).  Otherwise the SFU's sines, 2^-21 off, far below the rounding of 16 bits.
template <bool PRECISE>
__device__ __forceinline__ float2 cos_sin(float2 p, float2 f) {
    const float s = p.x * f.x, e = fmaf(p.x, f.x, -s), r = s - rintf(s);  // e, r: exact
    const float c = fmaf(p.x, f.y, fmaf(p.y, f.x, e)), a = r + c;
    float2 cs;
    if constexpr (PRECISE) {
        const float bb = a - r, lost = (r - (a - bb)) + (c - bb);  // r + c = a + lost (Knuth's two-sum)
        sincospif(2.f * a, &cs.y, &cs.x);
        const float d = 6.2831853071795865f * lost;
        return make_float2(fmaf(-d, cs.y, cs.x), fmaf(d, cs.x, cs.y));
    } else {
        __sincosf(6.2831853071795865f * a, &cs.y, &cs.x);
        return cs;
    }
}

// A head as `lanes` work units of two vectors, VE elements from `a` on and VE from `b`
// on (`two`: the second is there): first its rotation units, then the copied rest.
//   half layout (and one-element vectors): the two vectors' elements are partners.
//   interleaved, VE > 1: partners sit side by side in each of the two, which are half
//   the rotated part apart, as the copied ones are half the copied part apart.
template <int VE, bool PAIRED, bool INTERLEAVED> struct HeadMap {
    int rot_units, lanes, rot, tail, tail_units;
    __host__ __device__ __forceinline__ HeadMap(int Dh, int rot_) {
        rot = rot_;
        rot_units = PAIRED ? (rot / VE + 1) / 2 : rot / 2 / VE;
        tail = (Dh - rot) / VE;  // vectors
        tail_units = (tail + 1) / 2;
        lanes = rot_units + tail_units;
    }
    __device__ __forceinline__ void at(int l, int &a, int &b, bool &two) const {
        if (l < rot_units) {
            a = !PAIRED && INTERLEAVED ? 2 * l : l * VE;
            b = PAIRED ? a + rot_units * VE : INTERLEAVED ? a + 1 : a + rot / 2;
            two = !PAIRED || b < rot;
        } else {
            const int c = l - rot_units;
            a = rot + c * VE;
            b = a + tail_units * VE;
            two = c + tail_units < tail;
        }
    }
};

// float2 number m of a vector.
template <typename T> __device__ __forceinline__ float2 get_pair(const uint4 &v, int m) {
    if constexpr (sizeof(T) == 2) return Cvt<T>::unpack2(m == 0 ? v.x : m == 1 ? v.y : m == 2 ? v.z : v.w);
    else return m == 0 ? make_float2(__uint_as_float(v.x), __uint_as_float(v.y))
                       : make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
}
template <typename T> __device__ __forceinline__ float2 get_pair(uint32_t v, int) { return Cvt<T>::unpack2(v); }
template <typename T> __device__ __forceinline__ void put_pair(uint32_t &v, int, float2 f) {
    v = Cvt<T>::pack2(f.x, f.y);
}
template <typename T> __device__ __forceinline__ void put_pair(uint4 &v, int m, float2 f) {
    if constexpr (sizeof(T) == 2) {
        const uint32_t w = Cvt<T>::pack2(f.x, f.y);
        if (m == 0) v.x = w;
        else if (m == 1) v.y = w;
        else if (m == 2) v.z = w;
        else v.w = w;
    } else if (m == 0) {
        v.x = __float_as_uint(f.x);
        v.y = __float_as_uint(f.y);
    } else {
        v.z = __float_as_uint(f.x);
        v.w = __float_as_uint(f.y);
    }
}

// Heads whose loads a lane keeps in flight, two vectors each: with smaller vectors,
// more of them.
template <int VB> __host__ __device__ constexpr int heads_in_flight() { return VB == 16 ? 4 : 8; }

// wpt: warps a token, from token `whole` on (before it, one); cw: units of a head a
// warp takes at a time.
// APPEND: k and v go to cache rows.  AXES: each pair by the position of its axis.
template <typename T, int VB, bool INTERLEAVED, bool APPEND, bool AXES>
__global__ void __launch_bounds__(RX_NT, RX_CTAS_PER_SM) rope_ex_kernel(const __grid_constant__ RopeArgs<AXES> a,
                                                                       int64_t whole, int wpt, int cw) {
    using V = typename RawUnit<VB>::type;
    constexpr int VE = VB / (int)sizeof(T);
    constexpr bool PAIRED = INTERLEAVED && VE > 1;  // both halves of a pair in one vector
    constexpr int PP = VE;  // pairs a unit: float2 of cosines and of sines hold PP of them
    constexpr bool PRECISE = sizeof(T) == 4;
    constexpr int HB = heads_in_flight<VB>();
    __shared__ float2 s_turns[RX_MAX_DH / 2];
    const int half = a.rot / 2;
    __shared__ uint8_t s_axis[AXES ? RX_MAX_DH / 2 : 1];
    for (int i = threadIdx.x; i < half; i += RX_NT) {
        s_turns[i] = a.turns[i];
        if constexpr (AXES) s_axis[i] = a.axes.of[i];
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();

    // A warp covers `hpi` heads a step, a lane one unit of each head it meets: the
    // heads of q, then of k, then of v, which has no more units, all copied.
    const int lane = threadIdx.x & 31;
    const HeadMap<VE, PAIRED, INTERLEAVED> map(a.Dh, a.rot);
    const HeadMap<VE, PAIRED, INTERLEAVED> v_map(a.Dh, 0);
    const bool q_moves = a.q_out.p != a.q.p, k_moves = a.k_out.p != a.k.p;  // in place: nothing to copy
    const int hpi = 32 / cw, hs = lane / cw, lu = lane - hs * cw;
    const int n_qk = a.Hq + a.Hkv, n_all = n_qk + (APPEND ? a.Hkv : 0);
    const int64_t n_items = whole + (a.T - whole) * wpt, n_warps = (int64_t)gridDim.x * (RX_NT / 32);
    const int wshift = 31 - __clz(wpt);  // wpt is a power of two
    int64_t w = ((int64_t)blockIdx.x * RX_NT + threadIdx.x) >> 5;
    constexpr int NP = AXES ? RX_MAX_AXES : 1;
    int64_t p_next[NP] = {}, slot_next = 0;  // of the item ahead, loaded one item early
    auto token_of = [&](int64_t item) { return item < whole ? item : whole + ((item - whole) >> wshift); };
    auto look_ahead = [&](int64_t item) {
        if (item < n_items) {
            p_next[0] = a.positions[token_of(item)];
            if constexpr (AXES) {
#pragma unroll
                for (int x = 1; x < NP; ++x)
                    if (x < a.axes.n) p_next[x] = a.positions[x * a.T + token_of(item)];
            }
            if constexpr (APPEND) slot_next = a.slots[token_of(item)];
        }
    };
    look_ahead(w);
    for (; w < n_items; w += n_warps) {
        const int64_t t = token_of(w), slot = slot_next;
        float2 pos[NP] = {};
        bool pos_ok = true;
#pragma unroll
        for (int x = 0; x < NP; ++x) {
            if constexpr (AXES)
                if (x >= a.axes.n) break;
            pos[x] = split_position(p_next[x]);
            pos_ok = pos_ok && p_next[x] >= 0;
        }
        const int parts = w < whole ? 1 : wpt, part = w < whole ? 0 : (int)((w - whole) & (wpt - 1));
        look_ahead(w + n_warps);
        const int64_t b = a.S == a.T ? 0 : t / a.S, s = t - b * a.S;
        const bool slot_ok = !APPEND || slot < a.num_slots;
        if ((!pos_ok || !slot_ok) && lane == 0 && part == 0) atomicOr(a.status, BAD_INDEX);
        if (!pos_ok) continue;
        const int heads = !APPEND || (slot_ok && slot >= 0) ? n_all : a.Hq;
        // where heads 0 would be, counted through the list: q's, k's, v's
        auto place = [&](const Heads &x, int64_t row, bool batched, int before) {
            return (unsigned char *)x.p + ((batched ? b * x.sb + s * x.st : row * x.st) * (int64_t)sizeof(T) -
                                           (int64_t)before * x.head_bytes);
        };
        const unsigned char *q = place(a.q, 0, true, 0), *k = place(a.k, 0, true, a.Hq);
        const unsigned char *v = APPEND ? place(a.v, 0, true, n_qk) : nullptr;
        unsigned char *qo = place(a.q_out, 0, true, 0), *ko = place(a.k_out, slot, !APPEND, a.Hq);
        unsigned char *vo = APPEND ? place(a.v_out, slot, false, n_qk) : nullptr;
        auto head = [&](int h, const unsigned char *x0, const Heads &x, const unsigned char *y0, const Heads &y,
                        const unsigned char *z0, const Heads &z) {
            const unsigned char *base = h < a.Hq ? x0 : y0;
            uint32_t sh = h < a.Hq ? x.head_bytes : y.head_bytes;
            if (APPEND && h >= n_qk) {
                base = z0;
                sh = z.head_bytes;
            }
            return base + (uint64_t)(uint32_t)h * sh;
        };
        constexpr int PF = (PP + 1) / 2;
        float2 cs[PF], sn[PF];  // cosines and sines of the unit's pairs
        for (int u0 = 0; u0 < map.lanes; u0 += cw) {
            const int l = u0 + lu;
            if (l >= map.lanes || hs >= hpi) continue;
            int ia, ib, va, vb;
            bool two, v_two;
            map.at(l, ia, ib, two);
            v_map.at(l, va, vb, v_two);
            const bool turn = l < map.rot_units, copies_v = l < v_map.lanes;
            if (turn) {
#pragma unroll
                for (int m = 0; m < PP; ++m) {
                    // pairs of the first vector, then (PAIRED) of the second
                    const int pair = !PAIRED ? l * PP + m : m < PP / 2 ? ia / 2 + m : min(ib / 2 + m - PP / 2, half - 1);
                    float2 p = pos[0];
                    if constexpr (AXES) {
                        const int axis = s_axis[pair];
#pragma unroll
                        for (int i = 1; i < NP; ++i) p = axis == i ? pos[i] : p;
                    }
                    const float2 x = cos_sin<PRECISE>(p, s_turns[pair]);
                    const float cm = x.x * a.scale, sm = x.y * (a.scale * a.sign);
                    if (m & 1) {
                        cs[m / 2].y = cm;
                        sn[m / 2].y = sm;
                    } else {
                        cs[m / 2].x = cm;
                        sn[m / 2].x = sm;
                    }
                }
            }
            const int step = parts * hpi;
            // HB heads' loads ahead of their stores (heads never share an address, so
            // in place too)
            for (int h0 = part * hpi + hs; h0 < heads; h0 += HB * step) {
                V xa[HB], xb[HB];
                auto wanted = [&](int h) {
                    if (APPEND && h >= n_qk) return h < heads && (!PAIRED || copies_v);
                    return h < heads && (turn || (h < a.Hq ? q_moves : k_moves));
                };
#pragma unroll
                for (int j = 0; j < HB; ++j) {
                    const int h = h0 + j * step;
                    if (wanted(h)) {
                        const bool qk = !APPEND || h < n_qk;
                        const T *src = reinterpret_cast<const T *>(head(h, q, a.q, k, a.k, v, a.v));
                        xa[j] = *reinterpret_cast<const V *>(src + (qk ? ia : va));
                        if (qk ? two : v_two) xb[j] = *reinterpret_cast<const V *>(src + (qk ? ib : vb));
                    }
                }
#pragma unroll
                for (int j = 0; j < HB; ++j) {
                    const int h = h0 + j * step;
                    if (wanted(h)) {
                        if (turn && (!APPEND || h < n_qk)) {
                            // word by word, so that no vector is unpacked whole
                            constexpr int W = VB / 2 / (int)sizeof(T);  // float2 a vector
                            if constexpr (PAIRED) {                    // (a, b): one pair a float2
                                auto pairs = [&](V &x, int from) {
#pragma unroll
                                    for (int m = 0; m < W; ++m) {
                                        const float c = (from + m) & 1 ? cs[(from + m) / 2].y : cs[(from + m) / 2].x;
                                        const float s1 = (from + m) & 1 ? sn[(from + m) / 2].y : sn[(from + m) / 2].x;
                                        const float2 f = get_pair<T>(x, m);
                                        put_pair<T>(x, m, make_float2(fmaf(-f.y, s1, f.x * c), fmaf(f.x, s1, f.y * c)));
                                    }
                                };
                                pairs(xa[j], 0);
                                if (two) pairs(xb[j], W);
                            } else if constexpr (VE > 1) {  // two pairs: first elements in xa, second ones in xb
#pragma unroll
                                for (int m = 0; m < W; ++m) {
                                    const float2 f = get_pair<T>(xa[j], m), g = get_pair<T>(xb[j], m);
                                    const float2 fc = f2mul(f, cs[m]);
                                    put_pair<T>(xa[j], m, make_float2(fmaf(-g.x, sn[m].x, fc.x), fmaf(-g.y, sn[m].y, fc.y)));
                                    put_pair<T>(xb[j], m, f2fma(f, sn[m], f2mul(g, cs[m])));
                                }
                            } else {
                                float f[1], g[1], o[1], r[1];
                                unpack_unit<T, VB>(xa[j], f);
                                unpack_unit<T, VB>(xb[j], g);
                                o[0] = f[0] * cs[0].x - g[0] * sn[0].x;
                                r[0] = g[0] * cs[0].x + f[0] * sn[0].x;
                                xa[j] = pack_unit<T, VB>(o);
                                xb[j] = pack_unit<T, VB>(r);
                            }
                        }
                        const bool qk = !APPEND || h < n_qk;
                        T *dst = reinterpret_cast<T *>(const_cast<unsigned char *>(head(h, qo, a.q_out, ko, a.k_out, vo, a.v_out)));
                        *reinterpret_cast<V *>(dst + (qk ? ia : va)) = xa[j];
                        if (qk ? two : v_two) *reinterpret_cast<V *>(dst + (qk ? ib : vb)) = xb[j];
                    }
                }
            }
        }
    }
}

template <typename T, int VB, bool INTERLEAVED, bool AXES>
cudaError_t launch_layout(const RopeArgs<AXES> &a, int sm, cudaStream_t s) {
    constexpr int VE = VB / (int)sizeof(T);
    const int lanes = HeadMap<VE, (INTERLEAVED && VE > 1), INTERLEAVED>(a.Dh, a.rot).lanes;
    const RopePlan p = make_rope_plan(a.T, lanes, a.Hq + a.Hkv * (a.slots ? 2 : 1), heads_in_flight<VB>(),
                                      sm * RX_CTAS_PER_SM, RX_NT / 32);
    return launch_pdl(a.slots ? rope_ex_kernel<T, VB, INTERLEAVED, true, AXES> : rope_ex_kernel<T, VB, INTERLEAVED, false, AXES>,
                      dim3(p.grid), dim3(RX_NT), 0, s, a, p.whole, p.wpt, p.cw);
}

// unit: bytes that divide every address, stride and length.
template <typename T>
cudaError_t launch_type(const RopeArgs<false> &a, bool interleaved, int unit, int sm, cudaStream_t s) {
    if (unit == 16)
        return interleaved ? launch_layout<T, 16, true, false>(a, sm, s) : launch_layout<T, 16, false, false>(a, sm, s);
    if constexpr (sizeof(T) == 2)
        if (unit < 4)
            return interleaved ? launch_layout<T, 2, true, false>(a, sm, s) : launch_layout<T, 2, false, false>(a, sm, s);
    return interleaved ? launch_layout<T, 4, true, false>(a, sm, s) : launch_layout<T, 4, false, false>(a, sm, s);
}

}  // namespace rmsn
