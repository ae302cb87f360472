// norm_q8.h -- arguments of the 8-bit norm's kernels and how a call runs (the kernels
// are in norm_q8.cuh).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace rmsn {

struct Q8Args {
    const void *x, *res, *w;  // res null: none
    void *out, *nres;         // codes, one byte each; new residual
    float *scale;
    int64_t ld_x, ld_res, ld_out, ld_nres;
    int64_t rows;
    int64_t drop_row;       // test hook: this row's copy is never issued
    long long wait_budget;
    unsigned int *status;
    int D, group, groups;   // group: columns of a scale, 0: the row; groups a row
    int group_shift;        // log2(group)
    int whole_codes;        // a unit's codes are stored as one word
    int stages;
    uint32_t stage_bytes;   // of one tensor's row in the ring
    float eps, weight_bias;
};

// Q8_WARP, Q8_DIRECT and Q8_STAGED hold a row in registers, in 16-byte units: a row a
// warp, a row a CTA from global memory, a row a CTA from a ring.  Q8_LONG reads the row
// twice, in 16-byte units, Q8_GENERIC one element at a time.
enum : int { Q8_GENERIC = 0, Q8_WARP = 1, Q8_DIRECT = 2, Q8_STAGED = 3, Q8_LONG = 4 };

constexpr int Q8_GENERIC_NT = 512;
constexpr int Q8_WARP_NT = 256;
constexpr int Q8_UNITS = 4;     // Q8_STAGED: units a thread
constexpr int Q8_HEADER = 128;  // the ring's mbarriers
constexpr int Q8_MAX_STAGES = 8;
constexpr size_t Q8_SMEM_PER_SM = 228 * 1024;

struct Q8Plan {
    int kind, shift;       // shift: the rows' units are those of memory, their ends single elements
    int threads, units;    // units a thread
    int grid, stages;
    uint32_t stage_bytes;
    size_t smem;
};

// `classes`: 0: the row tensors stand differently to 16-byte boundaries; else they stand
// alike, a row `classes` rows on (1, 2, 4 or 8) like this one, 1 with `aligned`: on them.
inline Q8Plan make_q8_plan(int64_t rows, int64_t D, int es, bool residual, int64_t group, int classes, bool aligned, int sm) {
    Q8Plan p{};
    const int E = 16 / es;
    const int64_t units = D / E, row = D * es;
    p.shift = !(aligned && row % 16 == 0);
    auto two_passes = [&] {
        Q8Plan g{};
        g.kind = !p.shift && classes ? Q8_LONG : Q8_GENERIC;
        g.threads = Q8_GENERIC_NT;
        g.grid = (int)std::min<int64_t>(rows, 4 * (int64_t)sm);
        return g;
    };
    if (classes == 0 || units < 2 || units > 512 * Q8_UNITS) return two_passes();
    if (!p.shift && units <= 128) {
        p.kind = Q8_WARP;
        p.units = units <= 32 ? 1 : units <= 64 ? 2 : 4;
        int warps = Q8_WARP_NT / 32;  // rows side by side; fewer when SMs would idle
        while (warps > 1 && rows < (int64_t)warps * sm) warps /= 2;
        p.threads = 32 * warps;
        p.grid = (int)std::min<int64_t>((rows + warps - 1) / warps, (int64_t)sm * (512 / p.threads));
        return p;
    }
    auto threads_for = [&](int per) { return (int)(((units + per - 1) / per + 31) / 32 * 32); };
    const int threads = threads_for(Q8_UNITS);
    int per_sm = std::min(16, 512 / threads);  // at 128 registers a thread
    if (rows <= (int64_t)sm * per_sm) {
        p.kind = Q8_DIRECT;
        // One unit a thread has the shorter way through a row (4 x 4096: 2.1 us); two leave
        // room for more rows at once.
        p.units = units <= 512 && rows <= sm ? 1 : 2;
        p.threads = threads_for(p.units);
        p.grid = (int)rows;
        return p;
    }
    p.kind = Q8_STAGED;
    p.units = Q8_UNITS;
    p.threads = threads;
    p.stage_bytes = (uint32_t)((row + (p.shift ? 15 : 0) + 15) / 16 * 16);
    const size_t set = (size_t)(residual ? 2 : 1) * p.stage_bytes;
    // Two stages, or more while an SM's rings hold no more than 115 KB: deeper ones read
    // ahead at the cost of the writes (16384 rows of bf16 with residual, D = 8192: 148 us
    // with two, 152 with three; 6144: 110 and 118; 8192 without residual: 65.5, 64.0
    // with three, 67.7 with six).
    const size_t fixed = 1024 + 8 * 1024 + Q8_HEADER;  // of a CTA: the system's, static sums, barriers
    while (per_sm > 1 && Q8_SMEM_PER_SM / per_sm < fixed + 2 * set) --per_sm;
    const size_t room = Q8_SMEM_PER_SM / per_sm;
    if (room < fixed + 2 * set) return two_passes();
    p.stages = (int)std::min<size_t>({std::max<size_t>(2, 115 * 1024 / (set * per_sm)), (room - fixed) / set, (size_t)Q8_MAX_STAGES});
    // One, where four CTAs or more have 60 KB of rows under way with it, for many rows of
    // one scale each, which wait for memory alone (16384 x 4096: 73.0 us, 76.5 with two; x
    // 2048: 38.7 and 40.3; fp32 68.7 and 73.0; but 2560 with 50 KB 50.7 and 49.0, 2000 rows
    // of 4096 12.7 and 11.2, 8192 in groups of 128 42.3 and 40.4).
    if (per_sm >= 4 && set * per_sm >= 60 * 1024 && !group && !p.shift && rows >= 8 * (int64_t)sm * per_sm) p.stages = 1;
    p.smem = Q8_HEADER + (size_t)p.stages * set;
    p.grid = (int)std::min<int64_t>(rows, (int64_t)sm * per_sm);
    if (p.shift && classes > 1) {  // a CTA's rows all stand the same way
        p.grid = p.grid / classes * classes;
        if (p.grid == 0) return two_passes();
    }
    return p;
}

// Whether the kernels can run a plan (a launch of any other would leave its shared memory).
inline bool q8_plan_ok(const Q8Plan &p) {
    if (p.grid < 1 || p.threads < 32 || p.threads > 1024 || p.threads % 32) return false;
    if (p.kind == Q8_STAGED)
        return p.units == Q8_UNITS && p.threads <= 512 && p.stages >= 1 && p.stages <= Q8_MAX_STAGES && p.stage_bytes > 0;
    if (p.kind == Q8_WARP) return p.threads <= Q8_WARP_NT && !p.shift && (p.units == 1 || p.units == 2 || p.units == 4);
    if (p.kind == Q8_DIRECT) return p.units == 2 || (p.units == 1 && p.threads <= 512);
    return (p.kind == Q8_GENERIC || (p.kind == Q8_LONG && !p.shift)) && p.threads == Q8_GENERIC_NT;
}

// Launchers of one element type each (norm_q8_<type>.cu).
template <typename T> cudaError_t launch_q8(const Q8Plan &p, const Q8Args &a, cudaStream_t s);

}  // namespace rmsn
