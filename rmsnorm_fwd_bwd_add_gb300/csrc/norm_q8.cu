// norm_q8.cu -- rmsnorm_fwd_q8: the fused residual-add norm with an e4m3 output and its
// scales (argument checks and the choice of kernel; the plan is in norm_q8.h, the kernels in norm_q8.cuh).
#include "rmsnorm.h"

#include <algorithm>
#include <initializer_list>

#include "checks.h"
#include "common.cuh"
#include "norm_q8.h"

namespace rmsn {
int current_sm_count(int *sm);
int current_status_word(unsigned int **status);
void wait_settings(long long *budget, int64_t *drop);
int record_cuda_error(cudaError_t e);
}  // namespace rmsn

namespace {

using namespace rmsn;

// Whether a tensor's rows lie on 16-byte boundaries, or how many rows on they stand to
// them like the first again.
int classes_of(const Mat &m, int64_t rows, int es) {
    const int step = rows > 1 ? (int)((uint64_t)(m.ld * es) & 15u) : 0;
    int classes = 1;
    while (step * classes % 16) classes *= 2;
    return classes;
}
bool alike(const Mat &a, const Mat &b, int64_t rows, int es) {
    return (((uintptr_t)a.p ^ (uintptr_t)b.p) & 15u) == 0 && (rows <= 1 || (((a.ld - b.ld) * es) & 15) == 0);
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
    const int E = 16 / es;
    const bool together = !residual || (alike(mx, mr, rows, es) && alike(mx, mn, rows, es));
    const int classes = together ? classes_of(mx, rows, es) : 0;
    const bool on = rows_aligned(mx, es);
    // (weights are read in whole units where the rows' units are the columns')
    const Q8Plan p = make_q8_plan(rows, D, es, residual != nullptr, group, classes, on && aligned16(w), sm);
    Q8Args a{};
    a.x = x; a.ld_x = mx.ld;
    a.res = residual; a.ld_res = mr.ld;
    a.w = w;
    a.out = out; a.ld_out = mo.ld;
    a.nres = new_residual; a.ld_nres = mn.ld;
    a.scale = scale;
    a.rows = rows; a.D = (int)D;
    a.group = (int)group; a.groups = (int)groups;
    while (group && (1 << a.group_shift) < group) ++a.group_shift;
    a.eps = eps; a.weight_bias = weight_bias;
    a.stages = p.stages; a.stage_bytes = p.stage_bytes;
    // codes of a unit of x at a multiple of their number: the first row's, and each row's
    // step in codes like its step in elements of x
    const uintptr_t unit0 = (uintptr_t)out + (uintptr_t)(-((uintptr_t)x) & 15u) / es;
    a.whole_codes = unit0 % E == 0 && (rows <= 1 || (mo.ld - mx.ld) % E == 0);
    st = current_status_word(&a.status);
    if (st != RMSNORM_OK) return st;
    wait_settings(&a.wait_budget, &a.drop_row);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == RMSNORM_F16    ? launch_q8<__half>(p, a, s)
                          : dtype == RMSNORM_BF16 ? launch_q8<__nv_bfloat16>(p, a, s)
                                                  : launch_q8<float>(p, a, s);
    return e == cudaSuccess ? RMSNORM_OK : record_cuda_error(e);
}
