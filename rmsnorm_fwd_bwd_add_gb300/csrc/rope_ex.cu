// rope_ex.cu -- rotary positions for every head layout: half and interleaved
// pairs, part of the head, frequencies stretched for long contexts, tokens and
// heads a stride apart; forward, backward (the inverse rotation) and the append
// to the KV cache.
//
// A pair (a, b) of a head at position p becomes s (a cos t - b sin t, b cos t + a
// sin t), t = p * inv_freq; its VJP is the same with t negated, so one kernel
// serves both directions.  Elements past rot_dim are copied.
//
// Bound by memory: every element is read and written once.  A warp takes one
// token (or one of a token's parts, when tokens are fewer than warps): a lane
// owns one rotation unit -- the pairs of one vector (interleaved) or of two
// vectors half a rotation apart -- of 32 / units heads at a time and computes
// the cosines and sines of its pairs once for all of the token's heads.
//
// Angles are kept in turns (radians / 2 pi): the host splits inv_freq / 2 pi, in
// double, into a hi + lo pair of floats, the product with p is formed as a
// double-float, and the whole turns drop out exactly, so a position near 10^7
// still has its angle to about 1e-8 turns.  16-bit results take the SFU's sine
// and cosine of the reduced angle (2^-21 absolute, far below their rounding);
// fp32 results take sincospif.
#include "rmsnorm.h"

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "checks.h"
#include "common.cuh"
#include "launch_util.h"
#include "units.cuh"

namespace rmsn {
int current_sm_count(int *sm);
int current_status_word(unsigned int **status);
int record_cuda_error(cudaError_t e);
}  // namespace rmsn

namespace {

using namespace rmsn;

constexpr int RX_NT = 256;
constexpr int RX_CTAS_PER_SM = 2;
constexpr int RX_MAX_DH = 1024;
constexpr unsigned int BAD_INDEX = RMSNORM_DEVSTATUS_BAD_INDEX;

// One tensor [B, S, H, Dh]: strides in elements, Dh contiguous.
struct Heads {
    const void *p;
    int64_t sb, st, sh;
};

struct RopeExArgs {
    float2 turns[RX_MAX_DH / 2];  // (hi, lo) of inv_freq / 2 pi
    Heads q, k, v, q_out, k_out, v_out;
    const int64_t *positions, *slots;  // slots: null without a cache
    int64_t T, S, num_slots;
    int Hq, Hkv, Dh, rot;
    float scale, sign;
    unsigned int *status;
};

// (cos, sin) of p times a frequency in turns.
template <bool PRECISE>
__device__ __forceinline__ float2 cos_sin(int64_t p, float2 f) {
    const float ph = (float)p;
    const float pl = (float)(p - (int64_t)ph);
    const float s = ph * f.x;
    const float e = fmaf(ph, f.x, -s);  // exact error of that product
    float r = s - rintf(s);             // exact
    r += fmaf(ph, f.y, fmaf(pl, f.x, e));
    float2 cs;
    if constexpr (PRECISE) {
        sincospif(2.f * r, &cs.y, &cs.x);
    } else {
        __sincosf(6.2831853071795865f * r, &cs.y, &cs.x);
    }
    return cs;
}

// A head as `lanes` work units, each VE elements from `a` on and, where a unit has two
// vectors, VE more from `b` on: first its rotation units, then the copied rest.
//   interleaved, VE > 1: a rotation unit is one vector (VE / 2 pairs), a copied one too;
//   else: a rotation unit is two vectors whose elements are partners (half layout:
//   rot / 2 apart; one-element vectors: neighbours), a copied unit two vectors half
//   the copied part apart (the second may be past it).
template <int VE, bool PAIRED, bool INTERLEAVED> struct HeadMap {
    int rot_units, lanes, rest, tail, tail_units;
    __device__ __forceinline__ HeadMap(int Dh, int rot, bool copies) {
        rot_units = PAIRED ? rot / VE : rot / 2 / VE;
        rest = rot;
        tail = copies ? (Dh - rot) / VE : 0;  // vectors
        tail_units = PAIRED ? tail : (tail + 1) / 2;
        lanes = rot_units + tail_units;
    }
    __device__ __forceinline__ void at(int l, int &a, int &b, bool &two) const {
        if (l < rot_units) {
            a = PAIRED ? l * VE : INTERLEAVED ? 2 * l : l * VE;
            b = INTERLEAVED ? a + 1 : a + rest / 2;
            two = !PAIRED;
        } else {
            const int c = l - rot_units;
            a = rest + c * VE;
            b = a + tail_units * VE;
            two = !PAIRED && c + tail_units < tail;
        }
    }
};

// float2 number m of a 16-byte vector.
template <typename T> __device__ __forceinline__ float2 get_pair(const uint4 &v, int m) {
    if constexpr (sizeof(T) == 2) return Cvt<T>::unpack2(m == 0 ? v.x : m == 1 ? v.y : m == 2 ? v.z : v.w);
    else return m == 0 ? make_float2(__uint_as_float(v.x), __uint_as_float(v.y))
                       : make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
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

// Heads whose loads a lane keeps in flight: eight vectors.
template <bool PAIRED> __host__ __device__ constexpr int heads_in_flight() { return PAIRED ? 8 : 4; }

template <typename T, int VB, bool INTERLEAVED>
__global__ void __launch_bounds__(RX_NT, RX_CTAS_PER_SM) rope_ex_kernel(const __grid_constant__ RopeExArgs a,
                                                                       int wpt) {
    using V = typename RawUnit<VB>::type;
    constexpr int VE = VB / (int)sizeof(T);
    constexpr bool PAIRED = INTERLEAVED && VE > 1;  // both halves of a pair in one vector
    constexpr int PPU = PAIRED ? VE / 2 : VE;       // pairs a unit
    constexpr int PP = PAIRED || VE == 1 ? PPU : PPU / 2;  // float2 of cosines a unit
    constexpr bool PRECISE = sizeof(T) == 4;
    constexpr int HB = heads_in_flight<PAIRED>();
    __shared__ float2 s_turns[RX_MAX_DH / 2];
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < half; i += RX_NT) s_turns[i] = a.turns[i];
    __syncthreads();
    griddep_wait();

    // A warp covers `hpi` heads a step, a lane one unit of each head it meets: the
    // heads of q, then of k, then of v, which has as many units, all copied.
    const int lane = threadIdx.x & 31;
    const HeadMap<VE, PAIRED, INTERLEAVED> map(a.Dh, a.rot, true);
    const HeadMap<VE, PAIRED, INTERLEAVED> v_map(a.Dh, 0, true);
    const bool q_moves = a.q_out.p != a.q.p, k_moves = a.k_out.p != a.k.p;  // in place: nothing to copy
    const int hpi = map.lanes >= 32 ? 1 : 32 / map.lanes;
    const int hs = map.lanes >= 32 ? 0 : lane / map.lanes;
    const int n_qk = a.Hq + a.Hkv, n_all = n_qk + (a.slots ? a.Hkv : 0);
    const int64_t n_items = a.T * wpt, n_warps = (int64_t)gridDim.x * (RX_NT / 32);
    const int wshift = 31 - __clz(wpt);  // wpt is a power of two
    int64_t w = ((int64_t)blockIdx.x * RX_NT + threadIdx.x) >> 5;
    int64_t p_next = 0, slot_next = 0;  // of the item ahead, loaded one item early
    auto look_ahead = [&](int64_t item) {
        if (item < n_items) {
            p_next = a.positions[item >> wshift];
            if (a.slots) slot_next = a.slots[item >> wshift];
        }
    };
    look_ahead(w);
    for (; w < n_items; w += n_warps) {
        const int64_t t = w >> wshift, p = p_next, slot = slot_next;
        const int part = (int)(w & (wpt - 1));
        look_ahead(w + n_warps);
        const int64_t b = a.S == a.T ? 0 : t / a.S, s = t - b * a.S;
        const bool pos_ok = p >= 0, slot_ok = slot < a.num_slots;
        if ((!pos_ok || !slot_ok) && lane == 0 && part == 0) atomicOr(a.status, BAD_INDEX);
        if (!pos_ok) continue;
        const int heads = slot_ok && slot >= 0 ? n_all : a.Hq;
        // head h of its tensor is `stride` times h from its base
        const T *q = static_cast<const T *>(a.q.p) + b * a.q.sb + s * a.q.st;
        const T *k = static_cast<const T *>(a.k.p) + b * a.k.sb + s * a.k.st - a.Hq * a.k.sh;
        const T *v = static_cast<const T *>(a.v.p) + b * a.v.sb + s * a.v.st - n_qk * a.v.sh;
        T *qo = static_cast<T *>(const_cast<void *>(a.q_out.p)) + b * a.q_out.sb + s * a.q_out.st;
        T *ko = static_cast<T *>(const_cast<void *>(a.k_out.p)) +
                (a.slots ? slot * a.k_out.st : b * a.k_out.sb + s * a.k_out.st) - a.Hq * a.k_out.sh;
        T *vo = static_cast<T *>(const_cast<void *>(a.v_out.p)) + slot * a.v_out.st - n_qk * a.v_out.sh;
        float2 cs[PP], sn[PP];  // cosines and sines of the unit's pairs
        for (int u0 = 0; u0 < map.lanes; u0 += 32) {
            const int l = map.lanes >= 32 ? u0 + lane : lane - hs * map.lanes;
            if (l >= map.lanes || hs >= hpi) continue;
            int ia, ib, va, vb;
            bool two, v_two;
            map.at(l, ia, ib, two);
            v_map.at(l, va, vb, v_two);
            const bool turn = l < map.rot_units;
            if (turn) {
#pragma unroll
                for (int m = 0; m < PPU; ++m) {
                    const float2 x = cos_sin<PRECISE>(p, s_turns[l * PPU + m]);
                    const float cm = x.x * a.scale, sm = x.y * (a.scale * a.sign);
                    if constexpr (PAIRED || VE == 1) {
                        cs[m].x = cm;
                        sn[m].x = sm;
                    } else if (m & 1) {
                        cs[m / 2].y = cm;
                        sn[m / 2].y = sm;
                    } else {
                        cs[m / 2].x = cm;
                        sn[m / 2].x = sm;
                    }
                }
            }
            const int step = wpt * hpi;
            // HB heads' loads ahead of their stores (heads never share an address, so
            // in place too)
            for (int h0 = part * hpi + hs; h0 < heads; h0 += HB * step) {
                V xa[HB], xb[HB];
#pragma unroll
                for (int j = 0; j < HB; ++j) {
                    const int h = h0 + j * step;
                    if (h < heads && (turn || h >= n_qk || (h < a.Hq ? q_moves : k_moves))) {
                        const T *src = h < a.Hq ? q + h * a.q.sh : h < n_qk ? k + h * a.k.sh : v + h * a.v.sh;
                        xa[j] = *reinterpret_cast<const V *>(src + (h < n_qk ? ia : va));
                        if constexpr (!PAIRED)
                            if (h < n_qk ? two : v_two) xb[j] = *reinterpret_cast<const V *>(src + (h < n_qk ? ib : vb));
                    }
                }
#pragma unroll
                for (int j = 0; j < HB; ++j) {
                    const int h = h0 + j * step;
                    if (h < heads && (turn || h >= n_qk || (h < a.Hq ? q_moves : k_moves))) {
                        if (turn && h < n_qk) {
                            // word by word, so that no vector is unpacked whole
                            constexpr int W = sizeof(T) == 2 ? 4 : 2;  // float2 a vector
                            if constexpr (PAIRED) {                    // (a, b): one pair a float2
#pragma unroll
                                for (int m = 0; m < W; ++m) {
                                    const float2 f = get_pair<T>(xa[j], m);
                                    put_pair<T>(xa[j], m, make_float2(fmaf(-f.y, sn[m].x, f.x * cs[m].x),
                                                                      fmaf(f.x, sn[m].x, f.y * cs[m].x)));
                                }
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
                        T *dst = h < a.Hq ? qo + h * a.q_out.sh : h < n_qk ? ko + h * a.k_out.sh : vo + h * a.v_out.sh;
                        *reinterpret_cast<V *>(dst + (h < n_qk ? ia : va)) = xa[j];
                        if constexpr (!PAIRED)
                            if (h < n_qk ? two : v_two) *reinterpret_cast<V *>(dst + (h < n_qk ? ib : vb)) = xb[j];
                    }
                }
            }
        }
    }
    griddep_launch_dependents();
}

template <typename T, int VB>
cudaError_t launch_layout(const RopeExArgs &a, bool interleaved, int grid, int wpt, cudaStream_t s) {
    return interleaved ? launch_pdl(rope_ex_kernel<T, VB, true>, dim3(grid), dim3(RX_NT), 0, s, a, wpt)
                       : launch_pdl(rope_ex_kernel<T, VB, false>, dim3(grid), dim3(RX_NT), 0, s, a, wpt);
}

template <typename T>
cudaError_t launch_type(const RopeExArgs &a, bool interleaved, bool vec, int sm, cudaStream_t s) {
    // Warps a token.  Each of them computes the token's angles again, about half a
    // trip to memory, and makes a trip for every few heads; all warps go through
    // equal rounds of tokens' parts.
    const int64_t resident = (int64_t)sm * RX_CTAS_PER_SM, warps = resident * (RX_NT / 32);
    const int ve = vec ? 16 / (int)sizeof(T) : 1;
    const bool paired = interleaved && ve > 1;
    const int lanes = paired ? a.Dh / ve : (a.Dh / ve + 1) / 2, hpi = std::max(1, 32 / lanes);
    const int per_trip = hpi * (paired ? heads_in_flight<true>() : heads_in_flight<false>());
    const int heads = a.Hq + a.Hkv * (a.slots ? 2 : 1);
    int wpt = 1;
    int64_t best = INT64_MAX;
    for (int k = 1; k <= 8; k *= 2) {
        const int64_t rounds = (a.T * k + warps - 1) / warps, trips = (heads + per_trip * k - 1) / (per_trip * k);
        const int64_t cost = rounds * (1 + 2 * trips * ((lanes + 31) / 32));
        if (cost < best) {
            best = cost;
            wpt = k;
        }
    }
    const int grid = (int)std::min<int64_t>((a.T * wpt + RX_NT / 32 - 1) / (RX_NT / 32), resident);
    return vec ? launch_layout<T, 16>(a, interleaved, grid, wpt, s)
               : launch_layout<T, (int)sizeof(T)>(a, interleaved, grid, wpt, s);
}

// A [B, S, H, Dh] operand: whether its strides are usable, the bytes it spans,
// and for outputs that no two of its elements share an address.
struct Span {
    uintptr_t lo, hi;   // bytes [lo, hi)
    Mat m;              // as rows of one token (or one batch) each, a stride apart
    int64_t row;        // elements from such a row's first to its last, 0 if there is no such stride
};

bool safe_mul_add(int64_t n, int64_t st, int64_t *sum) {  // *sum += (n - 1) * st
    if (n > 1 && st > ((int64_t)1 << 60) / (n - 1)) return false;
    *sum += n > 1 ? (n - 1) * st : 0;
    return *sum < ((int64_t)1 << 60);
}

int span_of(const Heads &h, int64_t B, int64_t S, int64_t H, int64_t Dh, int es, bool output, Span *out) {
    *out = Span{0, 0, Mat{nullptr, 0}, 0};
    if (!h.p || B * S == 0 || H == 0) return RMSNORM_OK;
    if (!elem_aligned(h.p, es) || h.sb < 0 || h.st < 0 || h.sh < 0) return RMSNORM_ERR_INVALID_ARG;
    int64_t last = Dh - 1;
    if (!safe_mul_add(B, h.sb, &last) || !safe_mul_add(S, h.st, &last) || !safe_mul_add(H, h.sh, &last))
        return RMSNORM_ERR_UNSUPPORTED;
    if (output) {  // in order of stride, each dimension steps past the ones inside it
        struct { int64_t n, st; } d[3] = {{B, h.sb}, {S, h.st}, {H, h.sh}};
        std::sort(d, d + 3, [](auto &x, auto &y) { return x.st < y.st; });
        int64_t inner = Dh;
        for (auto &x : d) {
            if (x.n <= 1) continue;
            if (x.st < inner) return RMSNORM_ERR_INVALID_ARG;
            inner += (x.n - 1) * x.st;
        }
    }
    out->lo = (uintptr_t)h.p;
    out->hi = out->lo + (size_t)(last + 1) * es;
    const int64_t foot = (H - 1) * h.sh + Dh;
    const int64_t st = S > 1 ? h.st : h.sb;  // one stride from token to token
    if ((B == 1 || S == 1 || h.sb == S * h.st) && (B * S == 1 || st >= foot)) {
        out->m = mat(h.p, st, B * S, foot);
        out->row = foot;
    } else if (B > 1) {  // heads outside tokens: one stride from batch to batch
        const int64_t whole = (H - 1) * h.sh + (S - 1) * h.st + Dh;
        if (h.sb >= whole) {
            out->m = Mat{h.p, h.sb};
            out->row = whole;
        }
    }
    return RMSNORM_OK;
}

// Whether two operands may share a byte: by their rows where these are a common
// stride apart (heads of one fused projection), by whole spans otherwise.
bool spans_meet(const Span &a, const Span &b, int es) {
    if (a.hi <= b.lo || b.hi <= a.lo) return false;
    if (!a.row || !b.row || a.m.ld != b.m.ld) return true;
    const int64_t L = a.m.ld * es;
    int64_t r = (int64_t)(b.lo - a.lo) % L;
    if (r < 0) r += L;  // b's rows start r bytes into a's periods
    return r < a.row * es || r + b.row * es > L;
}

bool same_place(const Heads &a, const Heads &b, int64_t B, int64_t S, int64_t H) {
    return a.p == b.p && (B <= 1 || a.sb == b.sb) && (S <= 1 || a.st == b.st) && (H <= 1 || a.sh == b.sh);
}

bool vec_ok(const Heads &h, int64_t B, int64_t S, int64_t H, int es) {
    return !h.p || (aligned16(h.p) && (B <= 1 || h.sb * es % 16 == 0) && (S <= 1 || h.st * es % 16 == 0) &&
                    (H <= 1 || h.sh * es % 16 == 0));
}

Heads heads(const void *p, const int64_t *st, int n) {
    // n = 3: batch, token, head; n = 2: token, head
    return p && st ? Heads{p, n == 3 ? st[0] : 0, st[n - 2], st[n - 1]} : Heads{nullptr, 0, 0, 0};
}

// Checks, plans and launches; slots null: k_out has k's tokens.
int rope_run(const Heads &q, const Heads &k, const Heads &v, const int64_t *positions, const int64_t *slots,
             const Heads &q_out, const Heads &k_out, const Heads &v_out, const double *inv_freq,
             float attn_scale, int interleaved, int inverse, int64_t B, int64_t S, int64_t Hq, int64_t Hkv,
             int64_t Dh, int64_t rot, int64_t num_slots, int dtype, void *stream) {
    const int es = esize_of(dtype);
    const int64_t T = B * S;
    Span sq, sk, sv, sqo, sko, svo;
    int st = span_of(q, B, S, Hq, Dh, es, false, &sq);
    if (st == RMSNORM_OK) st = span_of(k, B, S, Hkv, Dh, es, false, &sk);
    if (st == RMSNORM_OK) st = span_of(v, B, S, Hkv, Dh, es, false, &sv);
    if (st == RMSNORM_OK) st = span_of(q_out, B, S, Hq, Dh, es, true, &sqo);
    const int64_t cb = slots ? 1 : B, cs = slots ? num_slots : S;
    if (st == RMSNORM_OK) st = span_of(k_out, cb, cs, Hkv, Dh, es, true, &sko);
    if (st == RMSNORM_OK) st = span_of(v_out, cb, cs, Hkv, Dh, es, true, &svo);
    if (st != RMSNORM_OK) return st;
    const bool q_in_place = same_place(q, q_out, B, S, Hq);
    const bool k_in_place = !slots && same_place(k, k_out, B, S, Hkv);
    // every output against every other operand
    if (!q_in_place && spans_meet(sqo, sq, es)) return RMSNORM_ERR_INVALID_ARG;
    if (!k_in_place && spans_meet(sko, sk, es)) return RMSNORM_ERR_INVALID_ARG;
    for (const Span *o : {&sko, &svo})
        if (spans_meet(*o, sq, es) || spans_meet(*o, sqo, es) || spans_meet(*o, sv, es))
            return RMSNORM_ERR_INVALID_ARG;
    if (spans_meet(sqo, sk, es) || spans_meet(sqo, sv, es) || spans_meet(svo, sk, es) ||
        spans_meet(sko, svo, es))
        return RMSNORM_ERR_INVALID_ARG;
    const size_t np = (size_t)T * 8;
    for (const Span *o : {&sqo, &sko, &svo})
        if (o->hi > o->lo && (overlaps((const void *)o->lo, o->hi - o->lo, positions, np) ||
                              overlaps((const void *)o->lo, o->hi - o->lo, slots, np)))
            return RMSNORM_ERR_INVALID_ARG;

    int sm = 0;
    unsigned int *status = nullptr;
    st = current_sm_count(&sm);
    if (st == RMSNORM_OK) st = current_status_word(&status);
    if (st != RMSNORM_OK) return st;
    static_assert(sizeof(RopeExArgs) < 8192, "kernel parameters stay small");
    RopeExArgs a;
    for (int i = 0; i < rot / 2; ++i) {
        const double f = inv_freq[i] * 0.15915494309189533576888;  // 1 / (2 pi)
        const float hi = (float)f;
        a.turns[i] = make_float2(hi, (float)(f - (double)hi));
    }
    a.q = q; a.k = k; a.v = v;
    a.q_out = q_out; a.k_out = k_out; a.v_out = v_out;
    a.positions = positions; a.slots = slots;
    a.T = T; a.S = S; a.num_slots = slots ? num_slots : INT64_MAX;
    a.Hq = (int)Hq; a.Hkv = (int)Hkv; a.Dh = (int)Dh; a.rot = (int)rot;
    a.scale = attn_scale;
    a.sign = inverse ? -1.f : 1.f;
    a.status = status;
    const int ve = 16 / es;
    const bool vec = (interleaved ? rot : rot / 2) % ve == 0 && Dh % ve == 0 && vec_ok(q, B, S, Hq, es) &&
                     vec_ok(q_out, B, S, Hq, es) && vec_ok(k, B, S, Hkv, es) && vec_ok(v, B, S, Hkv, es) &&
                     vec_ok(k_out, cb, cs, Hkv, es) && vec_ok(v_out, cb, cs, Hkv, es);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == RMSNORM_F16    ? launch_type<__half>(a, interleaved, vec, sm, s)
                          : dtype == RMSNORM_BF16 ? launch_type<__nv_bfloat16>(a, interleaved, vec, sm, s)
                                                  : launch_type<float>(a, interleaved, vec, sm, s);
    return e == cudaSuccess ? RMSNORM_OK : record_cuda_error(e);
}

// Shapes and scalars of both entry points.
int check_rope(const double *inv_freq, float attn_scale, int64_t B, int64_t S, int64_t Hq, int64_t Hkv,
               int64_t Dh, int64_t rot, int dtype) {
    if (dtype != RMSNORM_F16 && dtype != RMSNORM_BF16 && dtype != RMSNORM_F32) return RMSNORM_ERR_INVALID_ARG;
    if (B < 0 || S < 0 || Hq < 0 || Hkv < 0 || Dh <= 0 || rot <= 0 || rot % 2 || rot > Dh)
        return RMSNORM_ERR_INVALID_ARG;
    if (!inv_freq || !std::isfinite(attn_scale)) return RMSNORM_ERR_INVALID_ARG;
    if (Dh > RX_MAX_DH || Hq > (1 << 16) || Hkv > (1 << 16)) return RMSNORM_ERR_UNSUPPORTED;
    if (B > 0 && S > ((int64_t)1 << 40) / B) return RMSNORM_ERR_UNSUPPORTED;
    for (int64_t i = 0; i < rot / 2; ++i)
        if (!std::isfinite(inv_freq[i]) || std::fabs(inv_freq[i]) > 1e6) return RMSNORM_ERR_INVALID_ARG;
    return RMSNORM_OK;
}

}  // namespace

extern "C" int rmsnorm_rope(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                            const int64_t *positions, void *q_out, const int64_t *q_out_strides, void *k_out,
                            const int64_t *k_out_strides, const double *inv_freq, float attn_scale,
                            int interleaved, int inverse, int64_t B, int64_t S, int64_t Hq, int64_t Hkv,
                            int64_t Dh, int64_t rot_dim, int dtype, void *stream) {
    const int st = check_rope(inv_freq, attn_scale, B, S, Hq, Hkv, Dh, rot_dim, dtype);
    if (st != RMSNORM_OK) return st;
    if (B * S == 0 || Hq + Hkv == 0) return RMSNORM_OK;
    if (!positions || (Hq > 0 && (!q || !q_out || !q_strides || !q_out_strides)) ||
        (Hkv > 0 && (!k || !k_out || !k_strides || !k_out_strides)))
        return RMSNORM_ERR_INVALID_ARG;
    const Heads none{nullptr, 0, 0, 0};
    return rope_run(Hq ? heads(q, q_strides, 3) : none, Hkv ? heads(k, k_strides, 3) : none, none, positions,
                    nullptr, Hq ? heads(q_out, q_out_strides, 3) : none,
                    Hkv ? heads(k_out, k_out_strides, 3) : none, none, inv_freq, attn_scale, interleaved,
                    inverse, B, S, Hq, Hkv, Dh, rot_dim, 0, dtype, stream);
}

extern "C" int rmsnorm_rope_kv_append_ex(const void *q, const int64_t *q_strides, const void *k,
                                         const int64_t *k_strides, const void *v, const int64_t *v_strides,
                                         const int64_t *positions, const int64_t *slots, void *q_out,
                                         const int64_t *q_out_strides, void *k_cache,
                                         const int64_t *k_cache_strides, void *v_cache,
                                         const int64_t *v_cache_strides, const double *inv_freq,
                                         float attn_scale, int interleaved, int64_t T, int64_t Hq,
                                         int64_t Hkv, int64_t Dh, int64_t rot_dim, int64_t num_slots,
                                         int dtype, void *stream) {
    const int st = check_rope(inv_freq, attn_scale, 1, T, Hq, Hkv, Dh, rot_dim, dtype);
    if (st != RMSNORM_OK) return st;
    if (num_slots < 0) return RMSNORM_ERR_INVALID_ARG;
    if (T == 0 || Hq + Hkv == 0) return RMSNORM_OK;
    if (!positions || !slots || (Hq > 0 && (!q || !q_out || !q_strides || !q_out_strides)) ||
        (Hkv > 0 && (!k || !v || !k_strides || !v_strides || !k_cache_strides || !v_cache_strides ||
                     (num_slots > 0 && (!k_cache || !v_cache)))))
        return RMSNORM_ERR_INVALID_ARG;
    const Heads none{nullptr, 0, 0, 0};
    return rope_run(Hq ? heads(q, q_strides, 2) : none, Hkv ? heads(k, k_strides, 2) : none,
                    Hkv ? heads(v, v_strides, 2) : none, positions, slots,
                    Hq ? heads(q_out, q_out_strides, 2) : none, Hkv ? heads(k_cache, k_cache_strides, 2) : none,
                    Hkv ? heads(v_cache, v_cache_strides, 2) : none, inv_freq, attn_scale, interleaved, 0, 1, T,
                    Hq, Hkv, Dh, rot_dim, num_slots, dtype, stream);
}

extern "C" int rmsnorm_rope_frequencies(int scaling, int64_t rot_dim, double base, double factor,
                                        double trained_length, double low, double high, double *inv_freq,
                                        float *attn_scale) {
    const double two_pi = 6.283185307179586476925286766559;
    if (!inv_freq || !attn_scale || rot_dim <= 0 || rot_dim % 2) return RMSNORM_ERR_INVALID_ARG;
    if (rot_dim > RX_MAX_DH) return RMSNORM_ERR_UNSUPPORTED;
    if (!(base > 0) || !std::isfinite(base)) return RMSNORM_ERR_INVALID_ARG;
    if (scaling < RMSNORM_ROPE_PLAIN || scaling > RMSNORM_ROPE_LLAMA3) return RMSNORM_ERR_INVALID_ARG;
    if (scaling != RMSNORM_ROPE_PLAIN && (!(factor > 0) || !std::isfinite(factor))) return RMSNORM_ERR_INVALID_ARG;
    const bool banded = scaling == RMSNORM_ROPE_YARN || scaling == RMSNORM_ROPE_LLAMA3;
    if (banded && (!(trained_length > 0) || !std::isfinite(trained_length) || !(low > 0) || !(high > 0) ||
                   !std::isfinite(low) || !std::isfinite(high)))
        return RMSNORM_ERR_INVALID_ARG;
    if (scaling == RMSNORM_ROPE_LLAMA3 && !(high > low)) return RMSNORM_ERR_INVALID_ARG;
    if (scaling == RMSNORM_ROPE_YARN && (!(high >= low) || base == 1.0)) return RMSNORM_ERR_INVALID_ARG;
    if (scaling == RMSNORM_ROPE_NTK && rot_dim > 2)
        base *= std::pow(factor, (double)rot_dim / (double)(rot_dim - 2));
    *attn_scale = 1.f;
    double from = 0, to = 1;
    if (scaling == RMSNORM_ROPE_YARN) {
        // the pair that turns n times over the trained length, as an index
        auto pair_of = [&](double n) { return rot_dim * std::log(trained_length / (two_pi * n)) / (2 * std::log(base)); };
        from = std::max(std::floor(pair_of(high)), 0.0);
        to = std::min(std::ceil(pair_of(low)), (double)(rot_dim - 1));
        if (factor > 1) *attn_scale = (float)(0.1 * std::log(factor) + 1.0);
    }
    for (int64_t i = 0; i < rot_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * (double)i / (double)rot_dim);
        double keep = 1;  // share of the unstretched frequency
        if (scaling == RMSNORM_ROPE_LINEAR) keep = 0;
        if (scaling == RMSNORM_ROPE_YARN)
            keep = 1 - std::min(std::max(((double)i - from) / std::max(to - from, 1e-3), 0.0), 1.0);
        if (scaling == RMSNORM_ROPE_LLAMA3)
            keep = std::min(std::max((trained_length * f / two_pi - low) / (high - low), 0.0), 1.0);
        inv_freq[i] = keep == 1 ? f : f * keep + f / factor * (1 - keep);
    }
    return RMSNORM_OK;
}
