// block.cu -- rmsnorm_block_fwd and rmsnorm_block_vjp: the norms before and
// after a block fused with its gate and residual scale (argument checks and
// the choice of kernel; the kernels are in block_generic.cuh).
#include "rmsnorm.h"

#include <algorithm>
#include <cmath>

#include "block.h"
#include "block_generic.cuh"
#include "checks.h"
#include "launch_util.h"

namespace rmsn {
int current_sm_count(int *sm);
int current_status_word(unsigned int **status);
int record_cuda_error(cudaError_t e);
void wait_settings(long long *budget, int64_t *drop);
int scratch_alloc(size_t bytes, cudaStream_t s, void **out);
int scratch_free(void *p, cudaStream_t s);
}  // namespace rmsn

namespace {

using namespace rmsn;

template <typename T>
cudaError_t launch_fwd(const BlockArgs &a, int sm, cudaStream_t s) {
    const int grid = (int)std::min<int64_t>(a.rows, (int64_t)sm * 4);
    return launch_pdl(block_fwd_generic_kernel<T>, dim3(grid), dim3(BLOCK_GENERIC_NT), 0, s, a);
}

template <typename T>
cudaError_t launch_vjp(const BlockArgs &a, int grid, cudaStream_t s) {
    cudaError_t e = launch_pdl(block_vjp_generic_kernel<T>, dim3(grid), dim3(BLOCK_GENERIC_NT), 0, s, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(block_reduce_kernel<T>, dim3((unsigned)((a.D + 31) / 32)), dim3(32 * BR_WARPS), 0,
                      s, a, grid);
}

// What both directions check about the weights, the gate and the scale.
int check_block(const void *w_post, const void *w_pre, const void *gate, int64_t ld_gate,
                int64_t gate_rows, float scale, float eps, float weight_bias, int64_t rows, int64_t D,
                int dtype) {
    const int st = check_common(rows, D, dtype, eps, weight_bias);
    if (st != RMSNORM_OK) return st;
    const int es = esize_of(dtype);
    if (!w_pre || !std::isfinite(scale)) return RMSNORM_ERR_INVALID_ARG;
    if (!elem_aligned(w_pre, es) || !elem_aligned(w_post, es) || !elem_aligned(gate, es))
        return RMSNORM_ERR_INVALID_ARG;
    if (gate) {
        if (gate_rows <= 0 || rows % gate_rows) return RMSNORM_ERR_INVALID_ARG;
        if (gate_rows > INT64_MAX / (8 * D)) return RMSNORM_ERR_UNSUPPORTED;
        if (gate_rows > 1) return check_ld(ld_gate, gate_rows, D, es);
    }
    return RMSNORM_OK;
}

// The gate as a [G, D] matrix for the overlap checks.
Mat gate_mat(const void *gate, int64_t ld_gate, int64_t gate_rows, int64_t D) {
    return mat(gate, ld_gate, gate_rows, D);
}

bool mat_hits_gate(const Mat &m, int64_t rows, int64_t D, int es, const Mat &gate, int64_t gate_rows) {
    return mat_hits(m, rows, D, es, gate.p, extent(gate, gate_rows, D, es));
}

}  // namespace

extern "C" int rmsnorm_block_fwd(const void *y, int64_t ld_y, const void *residual, int64_t ld_residual,
                                 const void *w_post, const void *w_pre, const void *gate,
                                 int64_t ld_gate, int64_t gate_rows, float scale, float eps,
                                 float weight_bias, void *out, int64_t ld_out, void *new_residual,
                                 int64_t ld_new_residual, float *rstd, int64_t rows, int64_t D,
                                 int dtype, void *stream) {
    int st = check_block(w_post, w_pre, gate, ld_gate, gate_rows, scale, eps, weight_bias, rows, D, dtype);
    if (st != RMSNORM_OK) return st;
    if (rows == 0) return RMSNORM_OK;
    if (!y || !residual || !out || !new_residual) return RMSNORM_ERR_INVALID_ARG;
    const int es = esize_of(dtype);
    for (int64_t ld : {ld_y, ld_residual, ld_out, ld_new_residual}) {
        st = rows > 1 ? check_ld(ld, rows, D, es) : RMSNORM_OK;
        if (st != RMSNORM_OK) return st;
    }
    const Mat my = mat(y, ld_y, rows, D), mr = mat(residual, ld_residual, rows, D);
    const Mat mo = mat(out, ld_out, rows, D), mn = mat(new_residual, ld_new_residual, rows, D);
    const Mat mg = gate_mat(gate, ld_gate, gate_rows, D);
    for (const Mat *m : {&my, &mr, &mo, &mn})
        if (!elem_aligned(m->p, es)) return RMSNORM_ERR_INVALID_ARG;
    if (!elem_aligned(rstd, 4)) return RMSNORM_ERR_INVALID_ARG;
    const size_t nw = (size_t)D * es, nr = (size_t)rows * 8;
    if (mats_overlap(mo, mn, rows, D, es)) return RMSNORM_ERR_INVALID_ARG;
    for (const Mat *o : {&mo, &mn})
        if (bad_alias(*o, my, rows, D, es) || bad_alias(*o, mr, rows, D, es) ||
            mat_hits(*o, rows, D, es, w_post, nw) || mat_hits(*o, rows, D, es, w_pre, nw) ||
            mat_hits_gate(*o, rows, D, es, mg, gate_rows) || mat_hits(*o, rows, D, es, rstd, nr))
            return RMSNORM_ERR_INVALID_ARG;
    if (mat_hits(my, rows, D, es, rstd, nr) || mat_hits(mr, rows, D, es, rstd, nr) ||
        overlaps(rstd, nr, w_post, nw) || overlaps(rstd, nr, w_pre, nw) ||
        mat_hits(mg, gate_rows, D, es, rstd, nr))
        return RMSNORM_ERR_INVALID_ARG;

    int sm = 0;
    BlockArgs a{};
    st = current_sm_count(&sm);
    if (st == RMSNORM_OK) st = current_status_word(&a.status);
    if (st != RMSNORM_OK) return st;
    wait_settings(&a.wait_budget, &a.drop_row);
    a.y = y; a.ld_y = my.ld;
    a.res = residual; a.ld_res = mr.ld;
    a.w_post = w_post; a.w_pre = w_pre;
    a.gate = gate; a.ld_gate = mg.ld;
    a.rows_per_gate = gate ? rows / gate_rows : rows;
    a.out0 = out; a.ld_out0 = mo.ld;
    a.out1 = new_residual; a.ld_out1 = mn.ld;
    a.rstd = rstd;
    a.rows = rows; a.D = (int)D;
    a.eps = eps; a.weight_bias = weight_bias; a.scale = scale;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == RMSNORM_F16    ? launch_fwd<__half>(a, sm, s)
                          : dtype == RMSNORM_BF16 ? launch_fwd<__nv_bfloat16>(a, sm, s)
                                                  : launch_fwd<float>(a, sm, s);
    return e == cudaSuccess ? RMSNORM_OK : record_cuda_error(e);
}

extern "C" int rmsnorm_block_vjp(const void *y, int64_t ld_y, const void *h, int64_t ld_h,
                                 const void *w_post, const void *w_pre, const void *gate,
                                 int64_t ld_gate, int64_t gate_rows, float scale, const void *g_out,
                                 int64_t ld_g_out, const void *g_residual, int64_t ld_g_residual,
                                 const float *rstd, float eps, float weight_bias, void *g_y,
                                 int64_t ld_g_y, void *g_h, int64_t ld_g_h, float *gw_post,
                                 float *gw_pre, float *g_gate, int64_t rows, int64_t D, int dtype,
                                 void *stream) {
    int st = check_block(w_post, w_pre, gate, ld_gate, gate_rows, scale, eps, weight_bias, rows, D, dtype);
    if (st != RMSNORM_OK) return st;
    if (!gw_pre || (gw_post != nullptr) != (w_post != nullptr) || (g_gate != nullptr) != (gate != nullptr))
        return RMSNORM_ERR_INVALID_ARG;
    const int es = esize_of(dtype);
    if (!elem_aligned(gw_post, 4) || !elem_aligned(gw_pre, 4) || !elem_aligned(g_gate, 4) ||
        !elem_aligned(rstd, 4))
        return RMSNORM_ERR_INVALID_ARG;
    // the fp32 outputs against each other and every plain input
    const size_t nw = (size_t)D * es, ngw = (size_t)D * 4, nr = (size_t)rows * 8;
    const size_t ngg = gate ? (size_t)gate_rows * D * 4 : 0;
    const Mat mgate = gate_mat(gate, ld_gate, gate_rows, D);
    const size_t ngate = gate ? extent(mgate, gate_rows, D, es) : 0;
    const struct { const void *p; size_t n; } outs[] = {{gw_post, ngw}, {gw_pre, ngw}, {g_gate, ngg}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return RMSNORM_ERR_INVALID_ARG;
        if (overlaps(outs[i].p, outs[i].n, w_post, nw) || overlaps(outs[i].p, outs[i].n, w_pre, nw) ||
            overlaps(outs[i].p, outs[i].n, rstd, nr) || overlaps(outs[i].p, outs[i].n, gate, ngate))
            return RMSNORM_ERR_INVALID_ARG;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        for (const auto &o : outs) {
            const cudaError_t e = o.p ? cudaMemsetAsync(const_cast<void *>(o.p), 0, o.n, s) : cudaSuccess;
            if (e != cudaSuccess) return record_cuda_error(e);
        }
        return RMSNORM_OK;
    }
    if (!y || !h || !g_out || !g_y || !g_h) return RMSNORM_ERR_INVALID_ARG;
    const struct { const void *p; int64_t ld; } given[] = {{y, ld_y}, {h, ld_h}, {g_out, ld_g_out},
                                                          {g_residual, ld_g_residual}, {g_y, ld_g_y},
                                                          {g_h, ld_g_h}};
    Mat m[6];
    for (int i = 0; i < 6; ++i) {
        m[i] = mat(given[i].p, given[i].ld, rows, D);
        if (!given[i].p) continue;
        if (!elem_aligned(given[i].p, es)) return RMSNORM_ERR_INVALID_ARG;
        st = rows > 1 ? check_ld(given[i].ld, rows, D, es) : RMSNORM_OK;
        if (st != RMSNORM_OK) return st;
    }
    const Mat &mgy = m[4], &mgh = m[5];
    if (mats_overlap(mgy, mgh, rows, D, es)) return RMSNORM_ERR_INVALID_ARG;
    for (const Mat *o : {&mgy, &mgh}) {
        for (int i = 0; i < 4; ++i)
            if (m[i].p && bad_alias(*o, m[i], rows, D, es)) return RMSNORM_ERR_INVALID_ARG;
        if (mat_hits(*o, rows, D, es, w_post, nw) || mat_hits(*o, rows, D, es, w_pre, nw) ||
            mat_hits(*o, rows, D, es, rstd, nr) || mat_hits_gate(*o, rows, D, es, mgate, gate_rows))
            return RMSNORM_ERR_INVALID_ARG;
    }
    for (const Mat &x : m)
        for (const auto &o : outs)
            if (x.p && mat_hits(x, rows, D, es, o.p, o.n)) return RMSNORM_ERR_INVALID_ARG;

    int sm = 0;
    BlockArgs a{};
    st = current_sm_count(&sm);
    if (st == RMSNORM_OK) st = current_status_word(&a.status);
    if (st != RMSNORM_OK) return st;
    wait_settings(&a.wait_budget, &a.drop_row);
    a.y = y; a.ld_y = m[0].ld;
    a.res = h; a.ld_res = m[1].ld;
    a.g = g_out; a.ld_g = m[2].ld;
    a.g_res = g_residual; a.ld_g_res = m[3].ld;
    a.w_post = w_post; a.w_pre = w_pre;
    a.gate = gate; a.ld_gate = mgate.ld;
    a.rows_per_gate = gate ? rows / gate_rows : rows;
    a.out0 = g_y; a.ld_out0 = mgy.ld;
    a.out1 = g_h; a.ld_out1 = mgh.ld;
    a.rstd = const_cast<float *>(rstd);  // read only in the VJP kernels
    a.gw_post = gw_post; a.gw_pre = gw_pre; a.g_gate = g_gate;
    a.rows = rows; a.D = (int)D;
    a.eps = eps; a.weight_bias = weight_bias; a.scale = scale;
    // three fp32 rows of scratch a CTA: two CTAs an SM, fewer where the rows
    // are so long that they would take more than 256 MB
    const int64_t fit = ((int64_t)256 << 20) / (12 * D);
    const int grid = (int)std::min<int64_t>(rows, std::max<int64_t>(8, std::min<int64_t>(2 * sm, fit)));
    void *ws = nullptr;
    st = scratch_alloc((size_t)grid * D * 12, s, &ws);
    if (st != RMSNORM_OK) return st;
    a.part_pre = static_cast<float *>(ws);
    a.part_mid = a.part_pre + (size_t)grid * D;
    cudaError_t e = dtype == RMSNORM_F16    ? launch_vjp<__half>(a, grid, s)
                    : dtype == RMSNORM_BF16 ? launch_vjp<__nv_bfloat16>(a, grid, s)
                                            : launch_vjp<float>(a, grid, s);
    st = e == cudaSuccess ? RMSNORM_OK : record_cuda_error(e);
    const int freed = scratch_free(ws, s);
    return st != RMSNORM_OK ? st : freed;
}
