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
// fp32 results take sincospif, with the rounding of the reduced angle added to first order.
#include "rmsnorm.h"

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "checks.h"
#include "heads.h"
#include "rope_ex.cuh"
#include "rope_host.h"

namespace rmsn {
int current_sm_count(int *sm);
int current_status_word(unsigned int **status);
int record_cuda_error(cudaError_t e);

int rope_run(const Heads &q, const Heads &k, const Heads &v, const int64_t *positions, const PairAxes &axes,
             const int64_t *slots, const Heads &q_out, const Heads &k_out, const Heads &v_out,
             const double *inv_freq, float attn_scale, int interleaved, int inverse, int64_t B, int64_t S,
             int64_t Hq, int64_t Hkv, int64_t Dh, int64_t rot, int64_t num_slots, int dtype, void *stream) {
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
        if (o->hi > o->lo && (overlaps((const void *)o->lo, o->hi - o->lo, positions, np * axes.n) ||
                              overlaps((const void *)o->lo, o->hi - o->lo, slots, np)))
            return RMSNORM_ERR_INVALID_ARG;

    int sm = 0;
    unsigned int *status = nullptr;
    st = current_sm_count(&sm);
    if (st == RMSNORM_OK) st = current_status_word(&status);
    if (st != RMSNORM_OK) return st;
    static_assert(sizeof(RopeArgs<true>) < 8192, "kernel parameters stay small");
    RopeArgs<true> a;
    fill_rope_args(&a, q, k, v, positions, slots, q_out, k_out, v_out, inv_freq, attn_scale, inverse, T, S, Hq, Hkv,
                   Dh, rot, num_slots, status);
    fill_rope_axes(&a.axes, axes, rot);
    // the widest vectors that divide all of it, the rotated part's halves (half
    // layout) or whole (interleaved) and the head
    const uintptr_t bits = byte_bits(q, B, S, Hq, es) | byte_bits(q_out, B, S, Hq, es) |
                           byte_bits(k, B, S, Hkv, es) | byte_bits(v, B, S, Hkv, es) |
                           byte_bits(k_out, cb, cs, Hkv, es) | byte_bits(v_out, cb, cs, Hkv, es) |
                           (uintptr_t)((interleaved ? rot : rot / 2) * es) | (uintptr_t)(Dh * es);
    const int unit = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (axes.n > 1) {
        e = launch_rope_axes(a, interleaved, unit, dtype, sm, s);
    } else {
        RopeArgs<false> one;
        static_cast<RopeExArgs &>(one) = a;
        e = dtype == RMSNORM_F16    ? launch_type<__half>(one, interleaved, unit, sm, s)
            : dtype == RMSNORM_BF16 ? launch_type<__nv_bfloat16>(one, interleaved, unit, sm, s)
                                    : launch_type<float>(one, interleaved, unit, sm, s);
    }
    return e == cudaSuccess ? RMSNORM_OK : record_cuda_error(e);
}

}  // namespace rmsn

using namespace rmsn;

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
    return rope_run(Hq ? heads(q, q_strides, 3, es, Hq) : none, Hkv ? heads(k, k_strides, 3, es, Hkv) : none, none,
                    positions, PairAxes{}, nullptr, Hq ? heads(q_out, q_out_strides, 3, es, Hq) : none,
                    Hkv ? heads(k_out, k_out_strides, 3, es, Hkv) : none, none, inv_freq, attn_scale, interleaved,
                    inverse, B, S, Hq, Hkv, Dh, rot_dim, 0, dtype, stream);
}

extern "C" int rmsnorm_rope_axes(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                                 const int64_t *positions, int axes, const int32_t *pair_axis, void *q_out,
                                 const int64_t *q_out_strides, void *k_out, const int64_t *k_out_strides,
                                 const double *inv_freq, float attn_scale, int interleaved, int inverse, int64_t B,
                                 int64_t S, int64_t Hq, int64_t Hkv, int64_t Dh, int64_t rot_dim, int dtype,
                                 void *stream) {
    int st = check_rope(inv_freq, attn_scale, B, S, Hq, Hkv, Dh, rot_dim, dtype);
    if (st == RMSNORM_OK) st = check_axes(axes, pair_axis, rot_dim);
    if (st != RMSNORM_OK) return st;
    if (B * S == 0 || Hq + Hkv == 0) return RMSNORM_OK;
    if (!positions || (Hq > 0 && (!q || !q_out || !q_strides || !q_out_strides)) ||
        (Hkv > 0 && (!k || !k_out || !k_strides || !k_out_strides)))
        return RMSNORM_ERR_INVALID_ARG;
    const Heads none{nullptr, 0, 0, 0, 0};
    const int es = esize_of(dtype);
    return rope_run(Hq ? heads(q, q_strides, 3, es, Hq) : none, Hkv ? heads(k, k_strides, 3, es, Hkv) : none, none,
                    positions, PairAxes{axes, pair_axis}, nullptr, Hq ? heads(q_out, q_out_strides, 3, es, Hq) : none,
                    Hkv ? heads(k_out, k_out_strides, 3, es, Hkv) : none, none, inv_freq, attn_scale, interleaved,
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
    return rope_run(Hq ? heads(q, q_strides, 2, es, Hq) : none, Hkv ? heads(k, k_strides, 2, es, Hkv) : none,
                    Hkv ? heads(v, v_strides, 2, es, Hkv) : none, positions, PairAxes{}, slots,
                    Hq ? heads(q_out, q_out_strides, 2, es, Hq) : none,
                    Hkv ? heads(k_cache, k_cache_strides, 2, es, Hkv) : none,
                    Hkv ? heads(v_cache, v_cache_strides, 2, es, Hkv) : none, inv_freq, attn_scale, interleaved, 0, 1,
                    T, Hq, Hkv, Dh, rot_dim, num_slots, dtype, stream);
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
