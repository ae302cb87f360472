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
    float *part_post;              // VJP: [block_slices, D] sums of gw_post over runs of gate rows
    unsigned int *status;
    long long wait_budget;
    int64_t drop_row;              // test hook: this row's copy is never issued
    int64_t rows;
    int64_t rows_per_gate;         // rows / G (rows without a gate)
    int chunk_shift;               // rows are dealt out 2^chunk_shift at a time
    int team;                      // rows are dealt out (VJP: a gate row's to CTAs of their own)
    int64_t rows_per_team;         // VJP: rows_per_gate, or all rows where the gate has one for each
    int64_t split_q, split_r;      // team: CTAs / gate rows, else rows / CTAs, and the remainder
    int cluster;                   // VJP: the CTAs are one cluster, which adds up its own parts
    int run;                       // team: CTAs that share a run of rows (0: all of them)
    int64_t run_q, run_r;          // a team's rows / its runs, and the remainder
    float eps, weight_bias, scale;
    int D;
    int stages;
    uint32_t stage_bytes;          // of one tensor's row in the ring
};

// Part c of n things split into equal consecutive runs, the first n % parts of them
// one longer: q = n / parts and r = n % parts, divided once on the host.
__host__ __device__ inline int64_t split_first(int64_t c, int64_t q, int64_t r) { return c * q + (c < r ? c : r); }

// The part that has thing i.
template <typename I> __host__ __device__ inline I split_part(I i, I q, I r) {
    return i < r * (q + 1) ? i / (q + 1) : r + (i - r * (q + 1)) / q;
}

// row / rows_per_gate; 64-bit division costs a hundred instructions.
__host__ __device__ inline int64_t gate_row(int64_t row, int64_t rows_per_gate) {
    return (uint64_t)(row | rows_per_gate) >> 32 ? row / rows_per_gate : (uint32_t)row / (uint32_t)rows_per_gate;
}

// The rows of one CTA, in order.  They are dealt out to `size` CTAs in chunks of
// 2^shift: this one, `rank`, has rows lo + (k * size + rank) * 2^shift + j of [lo,
// hi).
struct RowDeal {
    int64_t lo, hi, n;  // n: how many rows
    int64_t rank, size;
    int shift;
    __host__ __device__ RowDeal(int64_t lo_, int64_t hi_, int64_t rank_, int64_t size_, int shift_)
        : lo(lo_), hi(hi_), rank(rank_), size(size_), shift(shift_) {
        const int64_t cycle = size << shift, full = gate_row(hi - lo, cycle);
        int64_t rest = (hi - lo) - full * cycle - (rank << shift);
        rest = rest < 0 ? 0 : rest < ((int64_t)1 << shift) ? rest : (int64_t)1 << shift;
        n = (full << shift) + rest;
    }
    __host__ __device__ int64_t row(int64_t i) const {
        return lo + ((((i >> shift) * size + rank) << shift) | (i & (((int64_t)1 << shift) - 1)));
    }
};

// Rows [lo, hi) of CTA `rank` of `size`: dealt out to all of them, or, with a.run, one
// of that many runs' to a.run CTAs each.
__host__ __device__ inline RowDeal team_rows(const BlockArgs &a, int64_t lo, int64_t hi, int64_t rank, int64_t size) {
    if (!a.run) return RowDeal(lo, hi, rank, size, a.chunk_shift);
    const int64_t g = (int64_t)((uint32_t)rank / (uint32_t)a.run);  // there are fewer than 2^31 CTAs
    return RowDeal(lo + split_first(g, a.run_q, a.run_r), lo + split_first(g + 1, a.run_q, a.run_r), rank - g * a.run,
                   a.run, 0);
}

// The forward's rows of CTA c.  team: dealt out to all CTAs; otherwise a run each.
__host__ __device__ inline RowDeal fwd_rows(const BlockArgs &a, int64_t c, int64_t grid) {
    if (a.team) return team_rows(a, 0, a.rows, c, grid);
    return RowDeal(split_first(c, a.split_q, a.split_r), split_first(c + 1, a.split_q, a.split_r), 0, 1, 0);
}

// The VJP's rows of CTA c.  team: the CTAs are split among the gate rows, and each
// gate row's rows dealt out to its CTAs (one gate row a CTA).  Otherwise CTA c has
// one run of rows, which may meet several gate rows.
__host__ __device__ inline RowDeal vjp_rows(const BlockArgs &a, int64_t c) {
    if (!a.team) {
        const int64_t r0 = split_first(c, a.split_q, a.split_r);
        return RowDeal(r0, split_first(c + 1, a.split_q, a.split_r), 0, 1, 0);
    }
    const int64_t q = a.split_q, r = a.split_r;
    const int64_t gr = (uint64_t)(c | q) >> 31 ? split_part<int64_t>(c, q, r)
                                                : (int64_t)split_part<uint32_t>((uint32_t)c, (uint32_t)q, (uint32_t)r);
    const int64_t c0 = split_first(gr, q, r);
    return team_rows(a, gr * a.rows_per_team, (gr + 1) * a.rows_per_team, c - c0, split_first(gr + 1, q, r) - c0);
}

// Where CTA c leaves its part of a gate row's sum A when it has not got all of
// that gate row's rows: at most its first and its last gate row are such, so two
// rows of part_mid a CTA hold them whatever the number of gate rows.
__host__ __device__ inline int64_t mid_slot(int64_t c, bool first) { return 2 * c + (first ? 0 : 1); }

// The second stage splits many gate rows into so many runs, a CTA each per 32
// columns: 5461 gate rows of 3 rows on 32 warps took 170 us of dependent trips to
// memory (D = 1000).
// Fewer of rows so long that the slices' sums would take more than 64 MB: their columns
// alone are thousands of CTAs.
constexpr int BLOCK_MAX_SLICES = 32;
inline int block_slices(int64_t gate_rows, int64_t D) {
    const int64_t most = ((int64_t)64 << 20) / (4 * D), n = gate_rows / 64 < most ? gate_rows / 64 : most;
    return gate_rows < 128 || n < 2 ? 1 : n < BLOCK_MAX_SLICES ? (int)n : BLOCK_MAX_SLICES;
}

// The ring of BLOCK_STAGED: its most stages, and the bytes of their mbarriers ahead
// of the table w1.
constexpr int BLOCK_MAX_STAGES = 8;
constexpr int BLOCK_HEADER = 128;

// Bytes of the table w1 in shared memory.
__host__ __device__ constexpr uint32_t block_table_bytes(int64_t D) { return ((uint32_t)D * 4u + 127u) & ~127u; }

// Bytes of a row of sums in shared memory.
__host__ __device__ constexpr size_t block_sum_bytes(int64_t D) { return (size_t)(D + 3) / 4 * 16; }

// How a call runs: BLOCK_GENERIC for rows that do not fit on chip, else the
// tier of block.cuh with units of `ub` bytes.
enum : int { BLOCK_STAGED = 0, BLOCK_DIRECT = 1, BLOCK_WARP = 2, BLOCK_GENERIC = 3 };

// What a VJP call has beside y, h and g.
enum : int { FORM_POST = 1, FORM_MORE = 2, FORM_SAVED = 4 };

struct BlockPlan {
    int kind, ub, threads, grid, stages, chunk_shift, team, half, shift, run, cluster;
    uint32_t stage_bytes;
    size_t smem;
};

// Launchers of one element type each (block_fwd_<type>.cu, block_vjp_<type>.cu).
template <typename T> cudaError_t launch_block_fwd(const BlockPlan &p, const BlockArgs &a, cudaStream_t s);
template <typename T> cudaError_t launch_block_vjp(const BlockPlan &p, const BlockArgs &a, cudaStream_t s);

}  // namespace rmsn
