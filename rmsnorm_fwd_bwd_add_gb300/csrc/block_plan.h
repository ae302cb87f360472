// block_plan.h -- how a call of the norm pair around a block runs: tier, unit, CTAs
// and shared memory from the sizes, alignment and operands (host only; the
// kernels are in block.cuh and block_generic.cuh, their instances in
// block_launch.cuh).
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "block.h"

namespace rmsn {

constexpr size_t BLOCK_SMEM_PER_SM = 227 * 1024;

// Threads an SM holds of the instance that CTAs of `threads` take (the register
// caps of block_launch.cuh).
inline int block_resident(int threads, bool vjp) {
    if (!vjp && ((threads > 256 && threads <= 320) || (threads > 512 && threads <= 640))) return 640;
    return threads > 512 ? 1024 : 512;
}

// Static shared memory of the widest instance that CTAs of `threads` take: its sums,
// two buffers of eight floats a warp.  Those of 641 threads or more (VJP: 513) take the
// one of 1024, the others one of at most 640.
inline size_t block_static_bytes(int threads, bool vjp, bool half) {
    return 64 * (threads > (vjp && !half ? 512 : 640) ? 1024 / 32 : 640 / 32);
}

// Picks tier, unit and grid.  `unit` divides every address and stride (16 at
// most); `tensors` row tensors are read.  `classes`: 0, or all row tensors stand
// alike to 16-byte boundaries, a row `classes` rows on (1, 2, 4 or 8) like this one.
inline BlockPlan make_block_plan(int64_t rows, int64_t D, int es, int unit, int tensors, bool vjp, int64_t gates, int sm,
                                 int classes) {
    BlockPlan p{};
    const int64_t row = D * es;
    p.ub = unit % 16 == 0 && row % 16 == 0 ? 16 : unit % 4 == 0 && row % 4 == 0 ? 4 : 2;
    const int per_thread = 32 / es;  // elements
    int64_t threads = ((D + per_thread - 1) / per_thread + 31) / 32 * 32;
    // Rows off 16-byte boundaries whose tensors stand alike: in the 16-byte units of
    // memory, the elements before the first and behind the last one a thread each (5000
    // rows of bf16, D = 4097: 49.6 us in 2-byte units, 28.7 so; VJP of 16384: 365 and
    // 159).  A CTA's rows all have to stand the same way: they are dealt out to a
    // multiple of `classes` CTAs.  Up to four units that would take a warp of their own
    // go the same way (VJP of 16384, D = 4104: 206 us with that warp, 160 without).
    int64_t units = row / 16;
    const bool few = units % 64 >= 1 && units % 64 <= 4;
    if (few) units -= units % 64;
    p.shift = classes > 0 && units > 64 && (p.ub < 16 || few);  // more than a warp's
    const int64_t width = p.shift ? units * (16 / es) : D;  // columns in units
    if (p.shift) threads = ((width + per_thread - 1) / per_thread + 31) / 32 * 32;
    // VJP rows of 257-320 threads leave an SM one CTA of 9 or 10 warps; with half as
    // much a thread it is 17 to 20 (16384 rows of bf16, D = 5120: 232 -> 207 us).
    if (vjp && threads > 256 && threads <= 320 && rows > sm) {
        p.half = 1;
        threads = ((width + per_thread / 2 - 1) / (per_thread / 2) + 31) / 32 * 32;
    }
    auto generic_plan = [&] {
        BlockPlan g{};
        g.kind = BLOCK_GENERIC;
        g.ub = p.ub;
        // as many CTAs as fit at once; the VJP keeps three fp32 rows of scratch each: fewer,
        // but eight, where they would take more than 256 MB (a CTA has a row at least, so it
        // is never more than the 12 bytes an element of the 16-bit row tensors)
        const int64_t fit = vjp ? std::max<int64_t>(8, ((int64_t)256 << 20) / (12 * D)) : 3 * sm;
        g.grid = (int)std::min<int64_t>(rows, std::min<int64_t>((vjp ? 2 : 3) * (int64_t)sm, fit));
        return g;
    };
    auto unshifted = [&] { return make_block_plan(rows, D, es, unit, tensors, vjp, gates, sm, 0); };
    p.ub = p.shift ? 16 : p.ub;
    if (threads > 1024) return p.shift ? unshifted() : generic_plan();
    p.threads = (int)threads;
    const size_t tables = block_table_bytes(D);
    // threads an SM holds of the instance these take (block_launch.cuh)
    const int resident = block_resident((int)threads, vjp);
    int per_sm = p.half ? 1 : resident / (int)threads;
    if (threads == 32) {
        p.kind = BLOCK_WARP;
        int warps = 8;  // rows side by side; fewer when the SMs would idle
        while (warps > 1 && rows < (int64_t)warps * sm) warps /= 2;
        // The VJP of few rows: all of them side by side in one cluster, which then adds
        // up their sums itself, in one launch and without scratch (64 rows of D = 512: 8.0
        // us a call instead of 10.8; the GPU takes 6.4 us, 7.2 in two stages).
        if (vjp && rows <= 64 && gates == 1) {
            warps = rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 ? 4 : 8;
            p.cluster = (int)((rows + warps - 1) / warps);
        }
        p.threads = 32 * warps;
        p.smem = vjp ? (size_t)(warps + (p.cluster ? 2 : 0)) * block_sum_bytes(D) : 0;
        p.grid = (int)std::min<int64_t>((rows + warps - 1) / warps, (int64_t)sm * (512 / p.threads));
        if (p.cluster) p.grid = p.cluster;
    } else if (rows <= (int64_t)sm * per_sm) {
        p.kind = BLOCK_DIRECT;
        p.grid = (int)rows;
        // as above, a row a CTA; two of them took longer than the second launch (16 rows
        // of D = 4096: 10.0 us of GPU time, 24 in two stages 8.2)
        if (vjp && rows <= 8) {
            p.cluster = p.grid;
            p.smem = 2 * block_sum_bytes(D);
        }
    } else {
        p.kind = BLOCK_STAGED;
        p.stage_bytes = (uint32_t)((row + (unit % 16 == 0 && row % 16 == 0 ? 0 : 15) + 15) / 16 * 16);
        // an SM's shared memory, less 1 KB a CTA for the system, its barriers and static
        // sums (2 KB at least) and its table; fewer CTAs where it would leave them no
        // second stage
        const size_t set = (size_t)tensors * p.stage_bytes;
        const size_t fixed = BLOCK_HEADER + block_static_bytes((int)threads, vjp, p.half);
        auto stages_of = [&](int ctas) {
            const size_t share = (BLOCK_SMEM_PER_SM + 1024) / ctas, used = 1024 + std::max<size_t>(2 * 1024, fixed) + tables;
            return share > used ? (int)std::min<size_t>(BLOCK_MAX_STAGES, (share - used) / set) : 0;
        };
        while (per_sm > 1 && stages_of(per_sm) < 2) --per_sm;
        p.stages = stages_of(per_sm);
        p.grid = (int)std::min<int64_t>(rows, (int64_t)sm * per_sm);
        p.smem = BLOCK_HEADER + tables + (size_t)p.stages * set;
        if (p.stages < 1) return p.shift ? unshifted() : generic_plan();
    }
    if (vjp && p.kind == BLOCK_WARP && !p.cluster)  // scratch traffic small beside the rows'
        p.grid = (int)std::min<int64_t>(p.grid, std::max<int64_t>(sm, rows / 12));
    if (vjp && p.kind == BLOCK_STAGED) {
        // A CTA's partial rows are 24 bytes a column, written and read in L2, a row 12
        // from and to memory: fewer rows a CTA the fewer its threads, whose waits
        // other CTAs must fill.
        const int64_t least = std::max<int64_t>(2, threads / 32);
        p.grid = (int)std::min<int64_t>(p.grid, std::max<int64_t>(sm, rows / least));
    }
    if (p.shift && classes > 1 && p.kind == BLOCK_STAGED) {
        const int64_t teams = vjp ? gates : 1, size = p.grid / teams / classes * classes;  // CTAs of a team
        if (size == 0) return unshifted();
        p.grid = (int)(size * teams);
        p.team = 1;
        p.run = row < 8192 ? classes : 0;
        return p;
    }
    // Rows of 8 KB or more are dealt out to the CTAs in turn, so that all of them work
    // on neighbouring memory: one row at a time in the VJP, 32 KB of them in the
    // forward while each CTA gets eight such chunks (16384 rows of bf16, D = 8192:
    // 183 us in one run a CTA, 169 dealt out singly, 166 in twos; 4096: 96, 91, and
    // 87 in fours; VJP 4096: 135.0 and 132.8).  Shorter rows lose by it (D = 1024:
    // 25 us in runs, 29 dealt out).  With a gate, its rows' CTAs must come out even
    // enough.
    p.team = p.kind != BLOCK_DIRECT && row >= 8192 && !(vjp && gates * 8 > p.grid);
    while (p.team && !vjp && (row << (p.chunk_shift + 1)) <= 32768 &&
           ((int64_t)p.grid << (p.chunk_shift + 1)) * 8 <= rows)
        ++p.chunk_shift;
    return p;
}

// The VJP's scratch: three fp32 rows a CTA, and one for each slice that the second
// stage may have, gates of two rows each being the most.
inline size_t block_scratch_bytes(int grid, int64_t rows, int64_t D) {
    const int slices = block_slices(rows / 2, D);
    return (((size_t)grid * 3 + (slices > 1 ? slices : 0)) * (size_t)D * 4 + 255) & ~(size_t)255;
}

// The most of it that any call of these sizes takes: rows on 16-byte boundaries, or off
// them and alike, with a gate that keeps them out of one cluster (no other plan has more
// CTAs).
inline size_t block_workspace_bytes(int64_t rows, int64_t D, int es, int sm) {
    return block_scratch_bytes(std::max(make_block_plan(rows, D, es, 16, 3, true, 2, sm, 0).grid,
                                        make_block_plan(rows, D, es, es, 3, true, 2, sm, 1).grid), rows, D);
}

// Whether the kernels can run a plan: a ring with stages to copy into, and rows off
// 16-byte boundaries on the tiers that take them.  A launch of any other would write
// outside its shared memory, so the launchers ask.
inline bool block_plan_ok(const BlockPlan &p) {
    if (p.grid < 1) return false;
    if (p.kind == BLOCK_GENERIC) return !p.shift && !p.cluster;
    if (p.threads < 32 || p.threads > 1024 || p.threads % 32) return false;
    if (p.kind == BLOCK_STAGED)
        return p.stages >= 1 && p.stages <= BLOCK_MAX_STAGES && p.stage_bytes > 0 && !p.cluster && (!p.half || p.threads <= 640);
    if (p.half || p.cluster < 0 || p.cluster > 8) return false;
    return p.kind == BLOCK_DIRECT || (p.kind == BLOCK_WARP && !p.shift && p.threads <= 256);
}

}  // namespace rmsn
