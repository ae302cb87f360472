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
constexpr int RX_HEADS = 4;  // heads whose loads a lane keeps in flight
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

// Interleaved layout: a unit is one vector (VE / 2 pairs); element kernels (VE =
// 1) take the pair as two vectors one apart.  Half layout: two vectors rot / 2
// apart (VE pairs).
template <typename T, int VB, bool INTERLEAVED>
__global__ void __launch_bounds__(RX_NT, RX_CTAS_PER_SM) rope_ex_kernel(const __grid_constant__ RopeExArgs a,
                                                                       int wpt) {
    using V = typename RawUnit<VB>::type;
    constexpr int VE = VB / (int)sizeof(T);
    constexpr bool PAIRED = INTERLEAVED && VE > 1;  // both halves of a pair in one vector
    constexpr int PPU = PAIRED ? VE / 2 : VE;       // pairs a unit
    constexpr bool PRECISE = sizeof(T) == 4;
    __shared__ float2 s_turns[RX_MAX_DH / 2];
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < half; i += RX_NT) s_turns[i] = a.turns[i];
    __syncthreads();
    griddep_wait();

    const int lane = threadIdx.x & 31;
    const int units = half / PPU;
    const int hpi = units >= 32 ? 1 : 32 / units;  // heads a warp covers a step
    const int hs = units >= 32 ? 0 : lane / units;
    const int H = a.Hq + a.Hkv;
    const int64_t n_items = a.T * wpt, n_warps = (int64_t)gridDim.x * (RX_NT / 32);
    for (int64_t w = ((int64_t)blockIdx.x * RX_NT + threadIdx.x) >> 5; w < n_items; w += n_warps) {
        const int64_t t = w / wpt;
        const int part = (int)(w - t * wpt);
        const int64_t b = a.S == a.T ? 0 : t / a.S, s = t - b * a.S;
        const int64_t p = a.positions[t];
        const int64_t slot = a.slots ? a.slots[t] : 0;
        const bool pos_ok = p >= 0, slot_ok = slot < a.num_slots;
        if ((!pos_ok || !slot_ok) && lane == 0 && part == 0) atomicOr(a.status, BAD_INDEX);
        if (!pos_ok) continue;
        const bool kv = slot_ok && slot >= 0;
        const int heads = kv ? H : a.Hq;  // q's, then k's
        const T *q = static_cast<const T *>(a.q.p) + b * a.q.sb + s * a.q.st;
        const T *k = static_cast<const T *>(a.k.p) + b * a.k.sb + s * a.k.st;
        T *qo = static_cast<T *>(const_cast<void *>(a.q_out.p)) + b * a.q_out.sb + s * a.q_out.st;
        T *ko = static_cast<T *>(const_cast<void *>(a.k_out.p)) +
                (a.slots ? slot * a.k_out.st : b * a.k_out.sb + s * a.k_out.st);
        auto src_of = [&](int h) -> const T * { return h < a.Hq ? q + h * a.q.sh : k + (h - a.Hq) * a.k.sh; };
        auto dst_of = [&](int h) -> T * { return h < a.Hq ? qo + h * a.q_out.sh : ko + (h - a.Hq) * a.k_out.sh; };

        for (int u0 = 0; u0 < units; u0 += 32) {
            const int u = units >= 32 ? u0 + lane : lane - hs * units;
            if (u >= units || hs >= hpi) continue;
            float2 cs[PPU];
#pragma unroll
            for (int m = 0; m < PPU; ++m) {
                cs[m] = cos_sin<PRECISE>(p, s_turns[u * PPU + m]);
                cs[m].x *= a.scale;
                cs[m].y *= a.scale * a.sign;
            }
            const int ia = PAIRED ? u * VE : INTERLEAVED ? 2 * u : u * VE;  // first element
            const int ib = INTERLEAVED ? ia + 1 : ia + half;                // its partner (not PAIRED)
            const int step = wpt * hpi;
            for (int h0 = part * hpi + hs; h0 < heads; h0 += RX_HEADS * step) {
                V xa[RX_HEADS], xb[RX_HEADS];
#pragma unroll
                for (int j = 0; j < RX_HEADS; ++j) {
                    const int h = h0 + j * step;
                    if (h < heads) {
                        const T *sp = src_of(h);
                        xa[j] = *reinterpret_cast<const V *>(sp + ia);
                        if constexpr (!PAIRED) xb[j] = *reinterpret_cast<const V *>(sp + ib);
                    }
                }
#pragma unroll
                for (int j = 0; j < RX_HEADS; ++j) {
                    const int h = h0 + j * step;
                    if (h < heads) {
                        T *dp = dst_of(h);
                        float fa[VE], fb[VE], ga[VE], gb[VE];
                        unpack_unit<T, VB>(xa[j], fa);
                        if constexpr (PAIRED) {
#pragma unroll
                            for (int m = 0; m < PPU; ++m) {
                                ga[2 * m] = fa[2 * m] * cs[m].x - fa[2 * m + 1] * cs[m].y;
                                ga[2 * m + 1] = fa[2 * m + 1] * cs[m].x + fa[2 * m] * cs[m].y;
                            }
                        } else {
                            unpack_unit<T, VB>(xb[j], fb);
#pragma unroll
                            for (int m = 0; m < PPU; ++m) {
                                ga[m] = fa[m] * cs[m].x - fb[m] * cs[m].y;
                                gb[m] = fb[m] * cs[m].x + fa[m] * cs[m].y;
                            }
                            *reinterpret_cast<V *>(dp + ib) = pack_unit<T, VB>(gb);
                        }
                        *reinterpret_cast<V *>(dp + ia) = pack_unit<T, VB>(ga);
                    }
                }
            }
        }
        // Vectors [c0, c1) of heads [h_lo, h_hi) copied unchanged.
        auto copy_heads = [&](auto from, auto to, int h_lo, int h_hi, int c0, int c1) {
            const int nv = c1 - c0;
            if (nv <= 0) return;
            const int chp = nv >= 32 ? 1 : 32 / nv;
            const int ch = nv >= 32 ? 0 : lane / nv;
            if (ch >= chp) return;
            for (int c = nv >= 32 ? lane : lane - ch * nv; c < nv; c += 32) {
                const int off = (c0 + c) * VE, step = wpt * chp;
                for (int h0 = h_lo + part * chp + ch; h0 < h_hi; h0 += RX_HEADS * step) {
                    V x[RX_HEADS];
#pragma unroll
                    for (int j = 0; j < RX_HEADS; ++j)
                        if (h0 + j * step < h_hi) x[j] = *reinterpret_cast<const V *>(from(h0 + j * step) + off);
#pragma unroll
                    for (int j = 0; j < RX_HEADS; ++j)
                        if (h0 + j * step < h_hi) *reinterpret_cast<V *>(to(h0 + j * step) + off) = x[j];
                }
            }
        };
        if (a.rot < a.Dh) {
            const bool q_moves = a.q_out.p != a.q.p, k_moves = a.k_out.p != a.k.p;
            copy_heads(src_of, dst_of, q_moves ? 0 : a.Hq, k_moves ? heads : a.Hq, a.rot / VE, a.Dh / VE);
        }
        if (a.slots && kv) {
            const T *v = static_cast<const T *>(a.v.p) + b * a.v.sb + s * a.v.st;
            T *vo = static_cast<T *>(const_cast<void *>(a.v_out.p)) + slot * a.v_out.st;
            copy_heads([&](int h) { return v + h * a.v.sh; }, [&](int h) { return vo + h * a.v_out.sh; }, 0,
                       a.Hkv, 0, a.Dh / VE);
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
    // warps a token: a few tokens are spread over up to eight warps each
    const int64_t resident = (int64_t)sm * RX_CTAS_PER_SM, warps = resident * (RX_NT / 32);
    const int wpt = (int)std::max<int64_t>(1, std::min<int64_t>(8, warps / a.T));
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
