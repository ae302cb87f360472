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
// token (or one of a token's parts, where tokens are fewer than warps): a lane
// owns one rotation unit -- the pairs of one vector (interleaved) or of two
// vectors half a rotation apart -- of 32 / units heads at a time and computes
// the cosines and sines of its pairs once for all of the token's heads.
//
// On the GB300, inputs changing from call to call: 16384 tokens of 32 + 8 heads of 128
// (bf16, views of one projection) 54.6 us, 92 % of the copy bandwidth; 5001 of 16 + 4 (fp32,
// interleaved, half rotated, inverse) 20.8 us, 73 %; the append of 4096 tokens of 32 + 8
// heads of 80 15.2 us, 62 % (on one set of buffers, which the L2 holds, 17.4 and 11.7);
// the append of 8 tokens 2.9 us of GPU time; 4096 tokens of 32 + 8 heads 17.7 us with heads of
// 128, 34.5 with heads of 126 (units of 4 bytes), 54.4 with heads of 125 (of 2).  The
// loops carry only loads, rotations and stores: every head's address is one 32 x 32 + 64
// multiply-add (64-bit strides cost a tenth of the time).
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
#include "rope_plan.h"
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

// One tensor [B, S, H, Dh]: strides in elements, Dh contiguous; and the head stride
// in bytes, below 2^32, so that a head's address is one multiply-add.
struct Heads {
    const void *p;
    int64_t sb, st, sh;
    uint32_t head_bytes;
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
// APPEND: k and v go to cache rows.
template <typename T, int VB, bool INTERLEAVED, bool APPEND>
__global__ void __launch_bounds__(RX_NT, RX_CTAS_PER_SM) rope_ex_kernel(const __grid_constant__ RopeExArgs a,
                                                                       int64_t whole, int wpt, int cw) {
    using V = typename RawUnit<VB>::type;
    constexpr int VE = VB / (int)sizeof(T);
    constexpr bool PAIRED = INTERLEAVED && VE > 1;  // both halves of a pair in one vector
    constexpr int PP = VE;  // pairs a unit: float2 of cosines and of sines hold PP of them
    constexpr bool PRECISE = sizeof(T) == 4;
    constexpr int HB = heads_in_flight<VB>();
    __shared__ float2 s_turns[RX_MAX_DH / 2];
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < half; i += RX_NT) s_turns[i] = a.turns[i];
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
    int64_t p_next = 0, slot_next = 0;  // of the item ahead, loaded one item early
    auto token_of = [&](int64_t item) { return item < whole ? item : whole + ((item - whole) >> wshift); };
    auto look_ahead = [&](int64_t item) {
        if (item < n_items) {
            p_next = a.positions[token_of(item)];
            if constexpr (APPEND) slot_next = a.slots[token_of(item)];
        }
    };
    look_ahead(w);
    for (; w < n_items; w += n_warps) {
        const int64_t t = token_of(w), p = p_next, slot = slot_next;
        const int parts = w < whole ? 1 : wpt, part = w < whole ? 0 : (int)((w - whole) & (wpt - 1));
        look_ahead(w + n_warps);
        const int64_t b = a.S == a.T ? 0 : t / a.S, s = t - b * a.S;
        const bool pos_ok = p >= 0, slot_ok = !APPEND || slot < a.num_slots;
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

template <typename T, int VB, bool INTERLEAVED>
cudaError_t launch_layout(const RopeExArgs &a, int sm, cudaStream_t s) {
    constexpr int VE = VB / (int)sizeof(T);
    const int lanes = HeadMap<VE, (INTERLEAVED && VE > 1), INTERLEAVED>(a.Dh, a.rot).lanes;
    const RopePlan p = make_rope_plan(a.T, lanes, a.Hq + a.Hkv * (a.slots ? 2 : 1), heads_in_flight<VB>(),
                                      sm * RX_CTAS_PER_SM, RX_NT / 32);
    return launch_pdl(a.slots ? rope_ex_kernel<T, VB, INTERLEAVED, true> : rope_ex_kernel<T, VB, INTERLEAVED, false>,
                      dim3(p.grid), dim3(RX_NT), 0, s, a, p.whole, p.wpt, p.cw);
}

// unit: bytes that divide every address, stride and length.
template <typename T>
cudaError_t launch_type(const RopeExArgs &a, bool interleaved, int unit, int sm, cudaStream_t s) {
    if (unit == 16) return interleaved ? launch_layout<T, 16, true>(a, sm, s) : launch_layout<T, 16, false>(a, sm, s);
    if constexpr (sizeof(T) == 2)
        if (unit < 4) return interleaved ? launch_layout<T, 2, true>(a, sm, s) : launch_layout<T, 2, false>(a, sm, s);
    return interleaved ? launch_layout<T, 4, true>(a, sm, s) : launch_layout<T, 4, false>(a, sm, s);
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
    if (H > 1 && h.sh > (int64_t)UINT32_MAX / es) return RMSNORM_ERR_UNSUPPORTED;
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

// The bits of every address and stride in bytes.
uintptr_t byte_bits(const Heads &h, int64_t B, int64_t S, int64_t H, int es) {
    if (!h.p) return 0;
    return (uintptr_t)h.p | (uintptr_t)((B > 1 ? h.sb : 0) * es) | (uintptr_t)((S > 1 ? h.st : 0) * es) |
           (uintptr_t)((H > 1 ? h.sh : 0) * es);
}

Heads heads(const void *p, const int64_t *st, int n, int es) {
    // n = 3: batch, token, head; n = 2: token, head
    return p && st ? Heads{p, n == 3 ? st[0] : 0, st[n - 2], st[n - 1], (uint32_t)(st[n - 1] * es)}
                   : Heads{nullptr, 0, 0, 0, 0};
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
    // the widest vectors that divide all of it, the rotated part's halves (half
    // layout) or whole (interleaved) and the head
    const uintptr_t bits = byte_bits(q, B, S, Hq, es) | byte_bits(q_out, B, S, Hq, es) |
                           byte_bits(k, B, S, Hkv, es) | byte_bits(v, B, S, Hkv, es) |
                           byte_bits(k_out, cb, cs, Hkv, es) | byte_bits(v_out, cb, cs, Hkv, es) |
                           (uintptr_t)((interleaved ? rot : rot / 2) * es) | (uintptr_t)(Dh * es);
    const int unit = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == RMSNORM_F16    ? launch_type<__half>(a, interleaved, unit, sm, s)
                          : dtype == RMSNORM_BF16 ? launch_type<__nv_bfloat16>(a, interleaved, unit, sm, s)
                                                  : launch_type<float>(a, interleaved, unit, sm, s);
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
    const Heads none{nullptr, 0, 0, 0, 0};
    const int es = esize_of(dtype);
    return rope_run(Hq ? heads(q, q_strides, 3, es) : none, Hkv ? heads(k, k_strides, 3, es) : none, none, positions,
                    nullptr, Hq ? heads(q_out, q_out_strides, 3, es) : none,
                    Hkv ? heads(k_out, k_out_strides, 3, es) : none, none, inv_freq, attn_scale, interleaved,
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
    const Heads none{nullptr, 0, 0, 0, 0};
    const int es = esize_of(dtype);
    return rope_run(Hq ? heads(q, q_strides, 2, es) : none, Hkv ? heads(k, k_strides, 2, es) : none,
                    Hkv ? heads(v, v_strides, 2, es) : none, positions, slots,
                    Hq ? heads(q_out, q_out_strides, 2, es) : none, Hkv ? heads(k_cache, k_cache_strides, 2, es) : none,
                    Hkv ? heads(v_cache, v_cache_strides, 2, es) : none, inv_freq, attn_scale, interleaved, 0, 1, T,
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
