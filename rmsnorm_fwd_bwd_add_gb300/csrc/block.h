// block.h -- what the kernels of the norm pair around a block share: their
// arguments and how their rows are split over the CTAs.
//
// Per row, with y the block's output, res the residual stream, w2 = weight_bias
// + w_post and w1 = weight_bias + w_pre (no w_post: r_y = w2 = 1):
//     r_y = 1 / sqrt(mean(y^2) + eps)
//     h   = res + scale * gate * (y * r_y * w2)          (new_residual)
//     r_h = 1 / sqrt(mean(h^2) + eps),  out = h * r_h * w1
// and its VJP, from g = the gradient of out and g_res = that of new_residual:
//     c    = r_h^2 * mean(g * w1 * h),  g_h = r_h * (g * w1 - h * c) + g_res
//     m    = scale * gate * w2
//     e    = r_y^2 * mean(m * g_h * y), g_y = r_y * (m * g_h - y * e)
//     A    = scale * sum over the rows of a gate row of g_h * y * r_y
//     g_gate = w2 * A,  gw_post = sum over gate rows of gate * A,
//     gw_pre = sum over rows of g * h * r_h
// One accumulator, A, thus serves the gate's and the post-norm weight's
// gradients alike.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rmsn {

struct BlockArgs {
    const void *y, *res;           // forward: residual; VJP: h, the new_residual it wrote
    const void *g, *g_res;         // VJP: gradients of out and of new_residual (or null)
    const void *w_post, *w_pre;    // w_post: null without a norm after the block
    const void *gate;              // [G, D], or null
    void *out0, *out1;             // forward: out, new_residual; VJP: g_y, g_h
    int64_t ld_y, ld_res, ld_g, ld_g_res, ld_gate, ld_out0, ld_out1;  // elements
    float *rstd;                   // [2, rows]: r_y, r_h (forward: written; VJP: read), or null
    float *g_gate;                 // VJP: [G, D], or null without a gate
    float *gw_post, *gw_pre;       // VJP: [D]
    float *part_pre;               // VJP: [grid, D] sums of g h r_h
    float *part_mid;               // VJP: [2 * grid, D] sums A of gate rows split over CTAs
    unsigned int *status;
    long long wait_budget;
    int64_t drop_row;              // test hook: this row's copy is never issued
    int64_t rows;
    int64_t rows_per_gate;         // rows / G (rows without a gate)
    float eps, weight_bias, scale;
    int D;
    int stages;
    uint32_t stage_bytes;          // of one tensor's row in the ring
};

// CTA c takes the consecutive rows [first_row(c), first_row(c + 1)), so a gate
// row's rows meet as few CTAs as they can and the sums over rows have a fixed
// order.
__host__ __device__ inline int64_t first_row(int64_t c, int64_t grid, int64_t rows) {
    const int64_t q = rows / grid, r = rows % grid;
    return c * q + (c < r ? c : r);
}

// The CTA that takes row i.
__host__ __device__ inline int64_t cta_of_row(int64_t i, int64_t grid, int64_t rows) {
    const int64_t q = rows / grid, r = rows % grid;
    return i < r * (q + 1) ? i / (q + 1) : r + (i - r * (q + 1)) / q;
}

// Where CTA c leaves its part of gate row gr's sum A when it has not got all
// of that gate row's rows: at most its first and its last gate row are such, so
// two rows of part_mid a CTA hold them whatever the number of gate rows.
__host__ __device__ inline int64_t mid_slot(int64_t c, int64_t gr, int64_t grid, int64_t rows,
                                            int64_t rows_per_gate) {
    return 2 * c + (gr != first_row(c, grid, rows) / rows_per_gate ? 1 : 0);
}

// How a call runs: BLOCK_GENERIC for rows that do not fit on chip, else the
// tier of block.cuh with units of `ub` bytes.
enum : int { BLOCK_STAGED = 0, BLOCK_DIRECT = 1, BLOCK_WARP = 2, BLOCK_GENERIC = 3 };

struct BlockPlan {
    int kind, ub, threads, grid, stages;
    uint32_t stage_bytes;
    size_t smem;
};

// Launchers of one element type each (block_fwd_<type>.cu, block_vjp_<type>.cu).
template <typename T> cudaError_t launch_block_fwd(const BlockPlan &p, const BlockArgs &a, cudaStream_t s);
template <typename T> cudaError_t launch_block_vjp(const BlockPlan &p, const BlockArgs &a, cudaStream_t s);

}  // namespace rmsn
