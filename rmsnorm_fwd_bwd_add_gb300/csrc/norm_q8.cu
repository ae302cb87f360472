// norm_q8.cu -- rmsnorm_fwd_q8: the fused residual-add norm with an e4m3 output and its
// scales (argument checks and the choice of kernel; the kernels are in norm_q8.cuh).
#include "rmsnorm.h"

#include <algorithm>
#include <initializer_list>

#include "checks.h"
#include "launch_util.h"
#include "norm_q8.cuh"

namespace rmsn {
int current_sm_count(int *sm);
int record_cuda_error(cudaError_t e);
}  // namespace rmsn

namespace {

using namespace rmsn;

template <typename T> cudaError_t launch_q8(const Q8Args &a, int sm, cudaStream_t s) {
    const dim3 grid((unsigned)std::min<int64_t>(a.rows, 4 * (int64_t)sm));
    return launch_pdl(a.res ? q8_generic_kernel<T, true> : q8_generic_kernel<T, false>, grid, dim3(Q8_GENERIC_NT), 0, s, a);
}

}  // namespace

extern "C" int rmsnorm_fwd_q8(const void *x, int64_t ld_x, const void *residual, int64_t ld_residual,
                              const void *w, float eps, float weight_bias, void *out, int64_t ld_out,
                              float *scale, int64_t group, void *new_residual, int64_t ld_new_residual,
                              int64_t rows, int64_t D, int dtype, void *stream) {
    int st = check_common(rows, D, dtype, eps, weight_bias);
    if (st != RMSNORM_OK) return st;
    if (group != 0 && group != 32 && group != 64 && group != 128) return RMSNORM_ERR_INVALID_ARG;
    if (!w || (residual == nullptr) != (new_residual == nullptr)) return RMSNORM_ERR_INVALID_ARG;
    if (rows == 0) return RMSNORM_OK;
    if (!x || !out || !scale) return RMSNORM_ERR_INVALID_ARG;
    const int es = esize_of(dtype);
    struct { int64_t ld; int es; bool used; } strides[] = {
        {ld_x, es, true}, {ld_residual, es, residual != nullptr}, {ld_new_residual, es, residual != nullptr}, {ld_out, 1, true}};
    for (const auto &l : strides)
        if (l.used && rows > 1) {
            st = check_ld(l.ld, rows, D, l.es);
            if (st != RMSNORM_OK) return st;
        }
    const Mat mx = mat(x, ld_x, rows, D), mr = mat(residual, ld_residual, rows, D);
    const Mat mo = mat(out, ld_out, rows, D), mn = mat(new_residual, ld_new_residual, rows, D);
    for (const Mat *m : {&mx, &mr, &mn})
        if (!elem_aligned(m->p, es)) return RMSNORM_ERR_INVALID_ARG;
    if (!elem_aligned(w, es) || !elem_aligned(scale, 4)) return RMSNORM_ERR_INVALID_ARG;
    const int64_t groups = group ? (D + group - 1) / group : 1;
    const size_t nw = (size_t)D * es, ns = (size_t)(rows * groups) * 4, no = extent(mo, rows, D, 1);
    if (bad_alias(mn, mx, rows, D, es) || bad_alias(mn, mr, rows, D, es)) return RMSNORM_ERR_INVALID_ARG;
    // codes, scales and new residual against each other and what is read
    if (overlaps(out, no, scale, ns) || overlaps(out, no, w, nw) || overlaps(scale, ns, w, nw) ||
        mat_hits(mn, rows, D, es, w, nw))
        return RMSNORM_ERR_INVALID_ARG;
    for (const Mat *m : {&mx, &mr, &mn})
        if (mat_hits(*m, rows, D, es, out, no) || mat_hits(*m, rows, D, es, scale, ns)) return RMSNORM_ERR_INVALID_ARG;

    int sm = 0;
    st = current_sm_count(&sm);
    if (st != RMSNORM_OK) return st;
    const Q8Args a{x,     residual, w,    out,    new_residual, scale, mx.ld, mr.ld,
                   mo.ld, mn.ld,    rows, (int)D, (int)group,   (int)groups, eps,   weight_bias};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == RMSNORM_F16    ? launch_q8<__half>(a, sm, s)
                          : dtype == RMSNORM_BF16 ? launch_q8<__nv_bfloat16>(a, sm, s)
                                                  : launch_q8<float>(a, sm, s);
    return e == cudaSuccess ? RMSNORM_OK : record_cuda_error(e);
}
