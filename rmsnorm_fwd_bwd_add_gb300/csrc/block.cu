// block.cu -- rmsnorm_block_fwd and rmsnorm_block_vjp: the norms before and
// after a block fused with its gate and residual scale (argument checks and
// the choice of kernel; the kernels are in block.cuh and block_generic.cuh).
#include "rmsnorm.h"

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "block.h"
#include "block_plan.h"
#include "common.cuh"
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

// The largest power of two up to 16 that divides the address and row stride.
int unit_of(const Mat &m, int64_t rows, int es) {
    if (!m.p) return 16;
    const uintptr_t bits = (uintptr_t)m.p | (rows > 1 ? (uintptr_t)(m.ld * es) : 0) | 16u;
    return (int)(bits & (~bits + 1));
}

// Whether the tensors' rows all stand alike to 16-byte boundaries: how many rows on
// they stand like the first again, or 0.
int classes_of(std::initializer_list<const Mat *> tensors, int64_t rows, int es) {
    int start = -1, step = 0;
    for (const Mat *m : tensors) {
        if (!m->p) continue;
        const int b = (int)((uintptr_t)m->p & 15u), d = rows > 1 ? (int)((uint64_t)(m->ld * es) & 15u) : 0;
        if (start >= 0 && (b != start || d != step)) return 0;
        start = b;
        step = d;
    }
    int classes = 1;
    while (step * classes % 16) classes *= 2;
    return classes;
}

// The runs of rows within a team.
void set_runs(BlockArgs *a, const BlockPlan &p, int64_t rows, int64_t size) {
    a->run = p.run;
    if (!p.run) return;
    a->run_q = rows / (size / p.run);
    a->run_r = rows % (size / p.run);
}

template <typename T> struct Tag { using type = T; };
template <typename F> auto by_type(int dtype, F f) {
    return dtype == RMSNORM_F16 ? f(Tag<__half>{}) : dtype == RMSNORM_BF16 ? f(Tag<__nv_bfloat16>{}) : f(Tag<float>{});
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
    if (gate && (rows || gate_rows)) {  // a gate row for each of no rows: none
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
    int unit = 16;
    for (const Mat *m : {&my, &mr, &mo, &mn}) unit = std::min(unit, unit_of(*m, rows, es));
    unit = std::min({unit, unit_of(mg, gate_rows, es), unit_of(Mat{w_pre, 0}, 1, es), unit_of(Mat{w_post, 0}, 1, es)});
    const bool per_row = gate && gate_rows == rows;
    const int classes = classes_of({&my, &mr, &mo, &mn, per_row ? &mg : &my}, rows, es);
    const BlockPlan p = make_block_plan(rows, D, es, unit, per_row ? 3 : 2, false, 1, sm, classes);
    a.stages = p.stages;
    a.stage_bytes = p.stage_bytes;
    a.chunk_shift = p.chunk_shift;
    a.team = p.team;
    a.split_q = rows / p.grid;
    a.split_r = rows % p.grid;
    set_runs(&a, p, rows, p.grid);
    const cudaError_t e = by_type(dtype, [&](auto t) { return launch_block_fwd<typename decltype(t)::type>(p, a, s); });
    return e == cudaSuccess ? RMSNORM_OK : record_cuda_error(e);
}

namespace {

// The VJP with its scratch in `workspace`, or, with `pooled`, from the library's pool.
int block_vjp(const void *y, int64_t ld_y, const void *h, int64_t ld_h, const void *w_post,
              const void *w_pre, const void *gate, int64_t ld_gate, int64_t gate_rows, float scale,
              const void *g_out, int64_t ld_g_out, const void *g_residual, int64_t ld_g_residual,
              const float *rstd, float eps, float weight_bias, void *g_y, int64_t ld_g_y, void *g_h,
              int64_t ld_g_h, float *gw_post, float *gw_pre, float *g_gate, int64_t rows, int64_t D,
              int dtype, bool pooled, void *workspace, size_t workspace_bytes, void *stream) {
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
    int unit = 16;
    for (const Mat &x : m) unit = std::min(unit, unit_of(x, rows, es));
    unit = std::min({unit, unit_of(mgate, gate_rows, es), unit_of(Mat{w_pre, 0}, 1, es),
                     unit_of(Mat{w_post, 0}, 1, es), unit_of(Mat{g_gate, 0}, 1, 4)});
    const bool per_row = gate && gate_rows == rows;
    const int64_t gates = gate && !per_row ? gate_rows : 1;  // gate rows with sums of their own
    const int classes = classes_of({&m[0], &m[1], &m[2], &m[3], &m[4], &m[5], per_row ? &mgate : &m[0]}, rows, es);
    const BlockPlan p = make_block_plan(rows, D, es, unit, 3 + (g_residual != nullptr) + per_row, true, gates, sm,
                                        classes);
    a.stages = p.stages;
    a.stage_bytes = p.stage_bytes;
    a.chunk_shift = p.chunk_shift;
    a.team = p.team;
    a.rows_per_team = rows / gates;
    a.split_q = p.team ? p.grid / gates : rows / p.grid;
    a.split_r = p.team ? p.grid % gates : rows % p.grid;
    set_runs(&a, p, a.rows_per_team, p.grid / gates);
    const size_t need = block_scratch_bytes(p.cluster ? 1 : p.grid, rows, D);
    void *ws = workspace;
    if (pooled && p.cluster) {
        ws = nullptr;  // nothing leaves the cluster
    } else if (pooled) {
        st = scratch_alloc(need, s, &ws);
        if (st != RMSNORM_OK) return st;
    } else {
        if (!ws || workspace_bytes < need || ((uintptr_t)ws & 255u)) return RMSNORM_ERR_INVALID_ARG;
        for (const Mat &x : m)
            if (x.p && mat_hits(x, rows, D, es, ws, need)) return RMSNORM_ERR_INVALID_ARG;
        for (const auto &o : outs)
            if (overlaps(o.p, o.n, ws, need)) return RMSNORM_ERR_INVALID_ARG;
        if (overlaps(ws, need, w_post, nw) || overlaps(ws, need, w_pre, nw) || overlaps(ws, need, rstd, nr) ||
            overlaps(ws, need, gate, ngate))
            return RMSNORM_ERR_INVALID_ARG;
    }
    a.cluster = p.cluster;
    if (ws) {
        a.part_pre = static_cast<float *>(ws);
        a.part_mid = a.part_pre + (size_t)p.grid * D;
        a.part_post = a.part_mid + 2 * (size_t)p.grid * D;
    }
    const cudaError_t e = by_type(dtype, [&](auto t) { return launch_block_vjp<typename decltype(t)::type>(p, a, s); });
    st = e == cudaSuccess ? RMSNORM_OK : record_cuda_error(e);
    const int freed = pooled && ws ? scratch_free(ws, s) : RMSNORM_OK;
    return st != RMSNORM_OK ? st : freed;
}

}  // namespace

#define BLOCK_VJP_PARAMS                                                                                    \
    const void *y, int64_t ld_y, const void *h, int64_t ld_h, const void *w_post, const void *w_pre,        \
        const void *gate, int64_t ld_gate, int64_t gate_rows, float scale, const void *g_out,               \
        int64_t ld_g_out, const void *g_residual, int64_t ld_g_residual, const float *rstd, float eps,      \
        float weight_bias, void *g_y, int64_t ld_g_y, void *g_h, int64_t ld_g_h, float *gw_post,            \
        float *gw_pre, float *g_gate, int64_t rows, int64_t D, int dtype
#define BLOCK_VJP_ARGS                                                                                      \
    y, ld_y, h, ld_h, w_post, w_pre, gate, ld_gate, gate_rows, scale, g_out, ld_g_out, g_residual,          \
        ld_g_residual, rstd, eps, weight_bias, g_y, ld_g_y, g_h, ld_g_h, gw_post, gw_pre, g_gate, rows, D,  \
        dtype

extern "C" int rmsnorm_block_vjp(BLOCK_VJP_PARAMS, void *stream) {
    return block_vjp(BLOCK_VJP_ARGS, true, nullptr, 0, stream);
}

extern "C" int rmsnorm_block_vjp_ws(BLOCK_VJP_PARAMS, void *workspace, size_t workspace_bytes, void *stream) {
    return block_vjp(BLOCK_VJP_ARGS, false, workspace, workspace_bytes, stream);
}

extern "C" size_t rmsnorm_block_vjp_workspace_size(int64_t rows, int64_t D, int dtype) {
    int sm = 0;
    if (check_common(rows, D, dtype, 0.f, 0.f) != RMSNORM_OK || rows == 0 || current_sm_count(&sm) != RMSNORM_OK)
        return 0;
    return block_workspace_bytes(rows, D, esize_of(dtype), sm);
}
