// kv_cache8.cu -- rmsnorm_kv_append and rmsnorm_kv_read: a KV cache of 8 bits with a scale
// a head, written and read back (argument checks and launches; the kernels are in
// kv_cache8.cuh).
#include "rmsnorm.h"

#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "checks.h"
#include "heads.h"
#include "kv_append8.h"
#include "kv_cache8.cuh"
#include "launch_util.h"
#include "rope_host.h"

namespace rmsn {
int current_sm_count(int *sm);
int current_status_word(unsigned int **status);
int record_cuda_error(cudaError_t e);
}  // namespace rmsn

namespace {

using namespace rmsn;

bool format_ok(int f) { return f == RMSNORM_CACHE_E4M3 || f == RMSNORM_CACHE_I8; }

Scales scales(const float *p, const int64_t *st) {
    return p && st ? Scales{const_cast<float *>(p), st[0], st[1]} : Scales{nullptr, 0, 0};
}

// The scales' extent, as heads of one element.
int span_of_scales(const Scales &c, int64_t N, int64_t H, bool output, Span *out) {
    return span_of(Heads{c.p, 0, c.st, c.sh, 0}, 1, N, H, 1, 4, output, out);
}

bool hits(const Span &a, const void *p, size_t n) {
    return a.hi > a.lo && overlaps((const void *)a.lo, a.hi - a.lo, p, n);
}

template <typename T, int FMT, int C> cudaError_t launch_read_units(const ReadArgs &a, int sm, cudaStream_t s) {
    const Read8Plan p = make_read8_plan(a.T, a.Dh / C, a.Hkv, sm, R8_CTAS_PER_SM, R8_SMALL_CTAS_PER_SM, C8_NT / 32);
    if (p.tokens > 1) return launch_pdl(read8_tokens_kernel<T, FMT, C>, dim3(p.grid), dim3(C8_NT), 0, s, a, p.cw, p.tokens);
    return launch_pdl(read8_kernel<T, FMT, C>, dim3(p.grid), dim3(C8_NT), 0, s, a, p.cw, p.wpt);
}

// unit: codes that divide every address, stride and head of the caches, and in
// elements those of the outputs.
template <typename T, int FMT> cudaError_t launch_read(const ReadArgs &a, int unit, int sm, cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (unit == 8) return launch_read_units<T, FMT, 8>(a, sm, s);
    return unit >= 4   ? launch_read_units<T, FMT, 4>(a, sm, s)
           : unit == 2 ? launch_read_units<T, FMT, 2>(a, sm, s)
                       : launch_read_units<T, FMT, 1>(a, sm, s);
}

template <typename T> struct Tag { using type = T; };
template <typename F> cudaError_t by_type(int dtype, int format, F f) {
    auto by_format = [&](auto t) {
        return format == RMSNORM_CACHE_I8 ? f(t, std::integral_constant<int, RMSNORM_CACHE_I8>{})
                                          : f(t, std::integral_constant<int, RMSNORM_CACHE_E4M3>{});
    };
    return dtype == RMSNORM_F16    ? by_format(Tag<__half>{})
           : dtype == RMSNORM_BF16 ? by_format(Tag<__nv_bfloat16>{})
                                   : by_format(Tag<float>{});
}

}  // namespace

extern "C" int rmsnorm_kv_append(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                                 const void *v, const int64_t *v_strides, const int64_t *positions, int axes,
                                 const int32_t *pair_axis, const int64_t *slots, void *q_out,
                                 const int64_t *q_out_strides, void *k_cache, const int64_t *k_cache_strides,
                                 void *v_cache, const int64_t *v_cache_strides, float *k_scale,
                                 const int64_t *k_scale_strides, float *v_scale, const int64_t *v_scale_strides,
                                 const double *inv_freq, float attn_scale, int interleaved, int64_t T, int64_t Hq,
                                 int64_t Hkv, int64_t Dh, int64_t rot_dim, int64_t num_slots, int cache_format,
                                 int dtype, void *stream) {
    int st = check_rope(inv_freq, attn_scale, 1, T, Hq, Hkv, Dh, rot_dim, dtype);
    if (st == RMSNORM_OK) st = check_axes(axes, pair_axis, rot_dim);
    if (st != RMSNORM_OK) return st;
    const bool same = cache_format == RMSNORM_CACHE_SAME;
    if (num_slots < 0 || (!same && !format_ok(cache_format))) return RMSNORM_ERR_INVALID_ARG;
    if (T == 0 || Hq + Hkv == 0) return RMSNORM_OK;
    if (!positions || !slots || (Hq > 0 && (!q || !q_out || !q_strides || !q_out_strides)) ||
        (Hkv > 0 && (!k || !v || !k_strides || !v_strides || !k_cache_strides || !v_cache_strides ||
                     (num_slots > 0 && (!k_cache || !v_cache)))))
        return RMSNORM_ERR_INVALID_ARG;
    if (same ? k_scale || v_scale
             : Hkv > 0 && num_slots > 0 && (!k_scale || !v_scale || !k_scale_strides || !v_scale_strides))
        return RMSNORM_ERR_INVALID_ARG;
    const Heads none{nullptr, 0, 0, 0, 0};
    const int es = esize_of(dtype), cs = same ? es : 1;
    const Heads hq = Hq ? heads(q, q_strides, 2, es, Hq) : none;
    const Heads hqo = Hq ? heads(q_out, q_out_strides, 2, es, Hq) : none;
    const Heads hk = Hkv ? heads(k, k_strides, 2, es, Hkv) : none, hv = Hkv ? heads(v, v_strides, 2, es, Hkv) : none;
    const Heads hkc = Hkv ? heads(k_cache, k_cache_strides, 2, cs, Hkv) : none;
    const Heads hvc = Hkv ? heads(v_cache, v_cache_strides, 2, cs, Hkv) : none;
    const PairAxes pair_axes{axes, pair_axis};
    if (same)
        return rope_run(hq, hk, hv, positions, pair_axes, slots, hqo, hkc, hvc, inv_freq, attn_scale, interleaved, 0, 1,
                        T, Hq, Hkv, Dh, rot_dim, num_slots, dtype, stream);
    const Scales ks = Hkv ? scales(k_scale, k_scale_strides) : Scales{nullptr, 0, 0};
    const Scales vs = Hkv ? scales(v_scale, v_scale_strides) : Scales{nullptr, 0, 0};

    Span sq, sk, sv, sqo, skc, svc, sks, svs;
    st = span_of(hq, 1, T, Hq, Dh, es, false, &sq);
    if (st == RMSNORM_OK) st = span_of(hk, 1, T, Hkv, Dh, es, false, &sk);
    if (st == RMSNORM_OK) st = span_of(hv, 1, T, Hkv, Dh, es, false, &sv);
    if (st == RMSNORM_OK) st = span_of(hqo, 1, T, Hq, Dh, es, true, &sqo);
    if (st == RMSNORM_OK) st = span_of(hkc, 1, num_slots, Hkv, Dh, 1, true, &skc);
    if (st == RMSNORM_OK) st = span_of(hvc, 1, num_slots, Hkv, Dh, 1, true, &svc);
    if (st == RMSNORM_OK) st = span_of_scales(ks, num_slots, Hkv, true, &sks);
    if (st == RMSNORM_OK) st = span_of_scales(vs, num_slots, Hkv, true, &svs);
    if (st != RMSNORM_OK) return st;
    if (!same_place(hq, hqo, 1, T, Hq) && spans_meet(sqo, sq, es)) return RMSNORM_ERR_INVALID_ARG;
    if (spans_meet(sqo, sk, es) || spans_meet(sqo, sv, es) || spans_meet(skc, svc, 1) || spans_meet(sks, svs, 4))
        return RMSNORM_ERR_INVALID_ARG;
    for (const Span *in : {&sq, &sk, &sv, &sqo})
        if (spans_meet(skc, 1, *in, es) || spans_meet(svc, 1, *in, es) || spans_meet(sks, 4, *in, es) ||
            spans_meet(svs, 4, *in, es))
            return RMSNORM_ERR_INVALID_ARG;
    for (const Span *o : {&sks, &svs})
        if (spans_meet(*o, 4, skc, 1) || spans_meet(*o, 4, svc, 1)) return RMSNORM_ERR_INVALID_ARG;
    const size_t np = (size_t)T * 8;
    for (const Span *o : {&sqo, &skc, &svc, &sks, &svs})
        if (hits(*o, positions, np * axes) || hits(*o, slots, np)) return RMSNORM_ERR_INVALID_ARG;

    int sm = 0;
    unsigned int *status = nullptr;
    st = current_sm_count(&sm);
    if (st == RMSNORM_OK) st = current_status_word(&status);
    if (st != RMSNORM_OK) return st;
    AppendArgs a;
    fill_rope_args(&a, hq, hk, hv, positions, slots, hqo, hkc, hvc, inv_freq, attn_scale, 0, T, T, Hq, Hkv, Dh,
                   rot_dim, num_slots, status);
    fill_rope_axes(&a.axes, pair_axes, rot_dim);
    a.k_scale = ks;
    a.v_scale = vs;
    // the widest vectors that divide the inputs, the rotated part's halves (half layout)
    // or whole (interleaved) and the head, with their codes at a multiple of their number
    const uintptr_t bits = byte_bits(hq, 1, T, Hq, es) | byte_bits(hqo, 1, T, Hq, es) | byte_bits(hk, 1, T, Hkv, es) |
                           byte_bits(hv, 1, T, Hkv, es) | byte_bits(hkc, 1, num_slots, Hkv, 1) * es |
                           byte_bits(hvc, 1, num_slots, Hkv, 1) * es |
                           (uintptr_t)((interleaved ? rot_dim : rot_dim / 2) * es) | (uintptr_t)(Dh * es);
    const int unit = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == RMSNORM_F16    ? launch_append8<__half>(a, cache_format, interleaved, unit, sm, s)
                          : dtype == RMSNORM_BF16 ? launch_append8<__nv_bfloat16>(a, cache_format, interleaved, unit, sm, s)
                                                  : launch_append8<float>(a, cache_format, interleaved, unit, sm, s);
    return e == cudaSuccess ? RMSNORM_OK : record_cuda_error(e);
}

extern "C" int rmsnorm_kv_read(const void *k_cache, const int64_t *k_cache_strides, const void *v_cache,
                               const int64_t *v_cache_strides, const float *k_scale, const int64_t *k_scale_strides,
                               const float *v_scale, const int64_t *v_scale_strides, const int64_t *slots,
                               void *k_out, const int64_t *k_out_strides, void *v_out, const int64_t *v_out_strides,
                               int64_t T, int64_t Hkv, int64_t Dh, int64_t num_slots, int cache_format, int dtype,
                               void *stream) {
    if (dtype != RMSNORM_F16 && dtype != RMSNORM_BF16 && dtype != RMSNORM_F32) return RMSNORM_ERR_INVALID_ARG;
    if (T < 0 || Hkv < 0 || Dh <= 0 || num_slots < 0 || !format_ok(cache_format)) return RMSNORM_ERR_INVALID_ARG;
    if (Dh > RX_MAX_DH || Hkv > (1 << 16) || T > ((int64_t)1 << 40)) return RMSNORM_ERR_UNSUPPORTED;
    if (T == 0 || Hkv == 0) return RMSNORM_OK;
    if (!slots || !k_out || !v_out || !k_out_strides || !v_out_strides) return RMSNORM_ERR_INVALID_ARG;
    if (num_slots > 0 && (!k_cache || !v_cache || !k_scale || !v_scale || !k_cache_strides || !v_cache_strides ||
                          !k_scale_strides || !v_scale_strides))
        return RMSNORM_ERR_INVALID_ARG;
    const int es = esize_of(dtype);
    const Heads hk = heads(k_cache, k_cache_strides, 2, 1, Hkv), hv = heads(v_cache, v_cache_strides, 2, 1, Hkv);
    const Heads hko = heads(k_out, k_out_strides, 2, es, Hkv), hvo = heads(v_out, v_out_strides, 2, es, Hkv);
    const Scales ks = scales(k_scale, k_scale_strides), vs = scales(v_scale, v_scale_strides);
    Span sk, sv, sks, svs, sko, svo;
    int st = span_of(hk, 1, num_slots, Hkv, Dh, 1, false, &sk);
    if (st == RMSNORM_OK) st = span_of(hv, 1, num_slots, Hkv, Dh, 1, false, &sv);
    if (st == RMSNORM_OK) st = span_of_scales(ks, num_slots, Hkv, false, &sks);
    if (st == RMSNORM_OK) st = span_of_scales(vs, num_slots, Hkv, false, &svs);
    if (st == RMSNORM_OK) st = span_of(hko, 1, T, Hkv, Dh, es, true, &sko);
    if (st == RMSNORM_OK) st = span_of(hvo, 1, T, Hkv, Dh, es, true, &svo);
    if (st != RMSNORM_OK) return st;
    if (spans_meet(sko, svo, es)) return RMSNORM_ERR_INVALID_ARG;
    for (const Span *o : {&sko, &svo})
        if (spans_meet(*o, es, sk, 1) || spans_meet(*o, es, sv, 1) || spans_meet(*o, es, sks, 4) ||
            spans_meet(*o, es, svs, 4) || hits(*o, slots, (size_t)T * 8))
            return RMSNORM_ERR_INVALID_ARG;
    int sm = 0;
    unsigned int *status = nullptr;
    st = current_sm_count(&sm);
    if (st == RMSNORM_OK) st = current_status_word(&status);
    if (st != RMSNORM_OK) return st;
    const ReadArgs a{hk, hv, hko, hvo, ks, vs, slots, T, num_slots, (int)Hkv, (int)Dh, status};
    // whole words of codes, and of elements: at most 16 bytes
    uintptr_t bits = (uintptr_t)Dh | byte_bits(hk, 1, num_slots, Hkv, 1) | byte_bits(hv, 1, num_slots, Hkv, 1);
    const uintptr_t out_bits = byte_bits(hko, 1, T, Hkv, es) | byte_bits(hvo, 1, T, Hkv, es);
    bits |= out_bits % 16 == 0 ? 0 : out_bits / es;
    const int unit = bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
    const cudaError_t e = by_type(dtype, cache_format, [&](auto t, auto f) {
        return launch_read<typename decltype(t)::type, decltype(f)::value>(a, unit, sm, static_cast<cudaStream_t>(stream));
    });
    return e == cudaSuccess ? RMSNORM_OK : record_cuda_error(e);
}
