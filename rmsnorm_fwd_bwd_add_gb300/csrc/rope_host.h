// rope_host.h -- what the rotary and cache entry points share on the host: the checks
// of shapes, scalars and axes, and the kernels' arguments.
#pragma once

#include <cmath>
#include <cstdint>

#include "heads.h"
#include "rope_ex.cuh"

namespace rmsn {

// The axis that each pair turns by; `of` null: one axis.
struct PairAxes {
    int n = 1;
    const int32_t *of = nullptr;
};

// Checks, plans and launches; slots null: k_out has k's tokens.
int rope_run(const Heads &q, const Heads &k, const Heads &v, const int64_t *positions, const PairAxes &axes,
             const int64_t *slots, const Heads &q_out, const Heads &k_out, const Heads &v_out,
             const double *inv_freq, float attn_scale, int interleaved, int inverse, int64_t B, int64_t S,
             int64_t Hq, int64_t Hkv, int64_t Dh, int64_t rot, int64_t num_slots, int dtype, void *stream);

// The instances of rope_axes.cu.
cudaError_t launch_rope_axes(const RopeArgs<true> &a, bool interleaved, int unit, int dtype, int sm, cudaStream_t s);

// Shapes and scalars.
inline int check_rope(const double *inv_freq, float attn_scale, int64_t B, int64_t S, int64_t Hq, int64_t Hkv,
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

inline int check_axes(int axes, const int32_t *pair_axis, int64_t rot) {
    if (axes < 1 || (axes > 1 && !pair_axis)) return RMSNORM_ERR_INVALID_ARG;
    if (axes > RMSNORM_ROPE_MAX_AXES) return RMSNORM_ERR_UNSUPPORTED;
    for (int64_t i = 0; pair_axis && i < rot / 2; ++i)
        if (pair_axis[i] < 0 || pair_axis[i] >= axes) return RMSNORM_ERR_INVALID_ARG;
    return RMSNORM_OK;
}

inline void fill_rope_args(RopeExArgs *a, const Heads &q, const Heads &k, const Heads &v, const int64_t *positions,
                           const int64_t *slots, const Heads &q_out, const Heads &k_out, const Heads &v_out,
                           const double *inv_freq, float attn_scale, int inverse, int64_t T, int64_t S, int64_t Hq,
                           int64_t Hkv, int64_t Dh, int64_t rot, int64_t num_slots, unsigned int *status) {
    for (int i = 0; i < rot / 2; ++i) {
        const double f = inv_freq[i] * 0.15915494309189533576888;  // 1 / (2 pi)
        const float hi = (float)f;
        a->turns[i] = make_float2(hi, (float)(f - (double)hi));
    }
    a->q = q; a->k = k; a->v = v;
    a->q_out = q_out; a->k_out = k_out; a->v_out = v_out;
    a->positions = positions; a->slots = slots;
    a->T = T; a->S = S; a->num_slots = slots ? num_slots : INT64_MAX;
    a->Hq = (int)Hq; a->Hkv = (int)Hkv; a->Dh = (int)Dh; a->rot = (int)rot;
    a->scale = attn_scale;
    a->sign = inverse ? -1.f : 1.f;
    a->status = status;
}

inline void fill_rope_axes(RopeAxes *a, const PairAxes &axes, int64_t rot) {
    a->n = axes.n;
    for (int64_t i = 0; i < rot / 2; ++i) a->of[i] = (uint8_t)(axes.of ? axes.of[i] : 0);
}

}  // namespace rmsn
