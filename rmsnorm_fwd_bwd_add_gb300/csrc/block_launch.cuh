// block_launch.cuh -- picks the instance of a block kernel for a plan.
#pragma once

#include "block.cuh"
#include "block_generic.cuh"
#include "block_plan.h"
#include "launch_util.h"

namespace rmsn {

cudaError_t launch_gw_reduce(const float *partials, float *gw, int P, int D, cudaStream_t stream);

template <bool VJP, typename T, int UB, int MAXT, int MINB, int KIND, bool GROW, bool SHIFT, int FORM = 0, bool HALF = false>
cudaError_t launch_block_inst(const BlockPlan &p, const BlockArgs &a, cudaStream_t s) {
    static std::atomic<uint64_t> smem_mask{0};
    void (*kern)(BlockArgs);
    if constexpr (VJP) kern = block_vjp_kernel<T, UB, MAXT, MINB, KIND, GROW, SHIFT, FORM, HALF>;
    else kern = block_fwd_kernel<T, UB, MAXT, MINB, KIND, GROW, SHIFT>;
    if (p.smem > 0) {
        const cudaError_t e = allow_max_dynamic_smem((const void *)kern, smem_mask);
        if (e != cudaSuccess) return e;
    }
    if constexpr (VJP && KIND != BLOCK_STAGED)
        if (p.cluster) return launch_pdl_cluster(kern, dim3(p.grid), dim3(p.threads), p.smem, s, p.cluster, a);
    return launch_pdl(kern, dim3(p.grid), dim3(p.threads), p.smem, s, a);
}

// The VJP's instances of one FORM, of rows of up to 512 threads.  Tests of what is there at
// run time cost a sixth of the instructions, and spills (16384 rows of bf16, D = 4096: without
// g_res 135 -> 117 us, without saved scales 151 -> 133, without post-norm 146 -> 132; D = 512
// 33.2 -> 28.1).  With a gate row per row they are compiled for saved scales, which a
// training backward has (fp32, 4095 x 2048, without g_res: 43.3 -> 41.1; bf16 without
// post-norm: 8192 x 4096 116.6 -> 107.7, 16384 x 512 40.1 -> 31.4), off 16-byte boundaries
// for all operands together; every other combination takes the instance that asks.
template <typename T, bool GROW, bool SHIFT, int FORM>
cudaError_t launch_block_form(const BlockPlan &p, const BlockArgs &a, cudaStream_t s) {
    if constexpr (!SHIFT)
        if (p.kind == BLOCK_WARP) return launch_block_inst<true, T, 16, 256, 2, BLOCK_WARP, GROW, false, FORM>(p, a, s);
    if (p.half) return launch_block_inst<true, T, 16, 640, 1, BLOCK_STAGED, GROW, SHIFT, FORM, true>(p, a, s);
    if (p.threads <= 256) return launch_block_inst<true, T, 16, 256, 2, BLOCK_STAGED, GROW, SHIFT, FORM>(p, a, s);
    return launch_block_inst<true, T, 16, 512, 1, BLOCK_STAGED, GROW, SHIFT, FORM>(p, a, s);
}

template <bool VJP, typename T, int UB, bool GROW, bool SHIFT>
cudaError_t launch_block_kind(const BlockPlan &p, const BlockArgs &a, cudaStream_t s) {
    if constexpr (VJP && UB == 16 && !(GROW && SHIFT))
        if (p.kind == BLOCK_WARP || (p.kind == BLOCK_STAGED && (p.half || p.threads <= 512))) {
            constexpr int ALL = FORM_POST | FORM_MORE | FORM_SAVED;
            const int form = (a.w_post ? FORM_POST : 0) | (a.g_res ? FORM_MORE : 0) | (a.rstd ? FORM_SAVED : 0);
            if (form == ALL) return launch_block_form<T, GROW, SHIFT, ALL>(p, a, s);
            if constexpr (GROW) {
                switch (form) {
                    case FORM_POST | FORM_SAVED: return launch_block_form<T, GROW, SHIFT, FORM_POST | FORM_SAVED>(p, a, s);
                    case FORM_MORE | FORM_SAVED: return launch_block_form<T, GROW, SHIFT, FORM_MORE | FORM_SAVED>(p, a, s);
                    case FORM_SAVED: return launch_block_form<T, GROW, SHIFT, FORM_SAVED>(p, a, s);
                    default: break;
                }
            } else if constexpr (!SHIFT) {
                switch (form) {
                    case FORM_POST | FORM_SAVED: return launch_block_form<T, GROW, SHIFT, FORM_POST | FORM_SAVED>(p, a, s);
                    case FORM_MORE | FORM_SAVED: return launch_block_form<T, GROW, SHIFT, FORM_MORE | FORM_SAVED>(p, a, s);
                    case FORM_SAVED: return launch_block_form<T, GROW, SHIFT, FORM_SAVED>(p, a, s);
                    case FORM_POST | FORM_MORE: return launch_block_form<T, GROW, SHIFT, FORM_POST | FORM_MORE>(p, a, s);
                    case FORM_POST: return launch_block_form<T, GROW, SHIFT, FORM_POST>(p, a, s);
                    case FORM_MORE: return launch_block_form<T, GROW, SHIFT, FORM_MORE>(p, a, s);
                    default: break;
                }
            }
        }
    if constexpr (!SHIFT)
        if (p.kind == BLOCK_WARP) return launch_block_inst<VJP, T, UB, 256, 2, BLOCK_WARP, GROW, false>(p, a, s);
    if (p.kind == BLOCK_DIRECT) {
        if (p.threads <= 512) return launch_block_inst<VJP, T, UB, 512, 1, BLOCK_DIRECT, GROW, SHIFT>(p, a, s);
        return launch_block_inst<VJP, T, UB, 1024, 1, BLOCK_DIRECT, GROW, SHIFT>(p, a, s);
    }
    if constexpr (VJP)
        if (p.half)  // at most 96 registers
            return launch_block_inst<VJP, T, UB, 640, 1, BLOCK_STAGED, GROW, SHIFT, 0, true>(p, a, s);
    // Threads an SM holds (block_resident): 512 with 128 registers each; the
    // forward also fits 96, so its CTAs of 257-320 threads sit two an SM and
    // those of 513-640 one.
    if (p.threads <= 256) return launch_block_inst<VJP, T, UB, 256, 2, BLOCK_STAGED, GROW, SHIFT>(p, a, s);
    if constexpr (!VJP)
        if (p.threads <= 320) return launch_block_inst<VJP, T, UB, 320, 2, BLOCK_STAGED, GROW, SHIFT>(p, a, s);
    if (p.threads <= 512) return launch_block_inst<VJP, T, UB, 512, 1, BLOCK_STAGED, GROW, SHIFT>(p, a, s);
    if constexpr (!VJP)
        if (p.threads <= 640) return launch_block_inst<VJP, T, UB, 640, 1, BLOCK_STAGED, GROW, SHIFT>(p, a, s);
    return launch_block_inst<VJP, T, UB, 1024, 1, BLOCK_STAGED, GROW, SHIFT>(p, a, s);
}

template <bool VJP, typename T, int UB, bool SHIFT = false>
cudaError_t launch_block_unit(const BlockPlan &p, const BlockArgs &a, cudaStream_t s) {
    return a.gate && a.rows_per_gate == 1 ? launch_block_kind<VJP, T, UB, true, SHIFT>(p, a, s)
                                          : launch_block_kind<VJP, T, UB, false, SHIFT>(p, a, s);
}

template <bool VJP, typename T, int UB>
cudaError_t launch_block_generic(const BlockPlan &p, const BlockArgs &a, cudaStream_t s) {
    return launch_pdl(VJP ? block_vjp_generic_kernel<T, UB> : block_fwd_generic_kernel<T, UB>, dim3(p.grid),
                      dim3(BLOCK_GENERIC_NT), 0, s, a);
}

template <bool VJP, typename T>
cudaError_t launch_block(const BlockPlan &p, const BlockArgs &a, cudaStream_t s) {
    if (!block_plan_ok(p)) return cudaErrorInvalidConfiguration;
    if (p.kind == BLOCK_GENERIC)
        return p.ub == 16 ? launch_block_generic<VJP, T, 16>(p, a, s) : launch_block_generic<VJP, T, sizeof(T)>(p, a, s);
    if (p.shift) return launch_block_unit<VJP, T, 16, true>(p, a, s);
    if (p.ub == 16) return launch_block_unit<VJP, T, 16>(p, a, s);
    if constexpr (sizeof(T) == 2)
        if (p.ub == 2) return launch_block_unit<VJP, T, 2>(p, a, s);
    return launch_block_unit<VJP, T, 4>(p, a, s);
}

template <typename T, int W>
cudaError_t launch_block_reduce(const BlockPlan &p, const BlockArgs &a, int slices, cudaStream_t s) {
    const dim3 grid((unsigned)((a.D + 31) / 32), slices), block(32 * W);
    return a.rows <= INT32_MAX ? launch_pdl(block_reduce_kernel<T, uint32_t, W>, grid, block, 0, s, a, p.grid)
                               : launch_pdl(block_reduce_kernel<T, int64_t, W>, grid, block, 0, s, a, p.grid);
}

template <typename T>
cudaError_t launch_block_vjp_both(const BlockPlan &p, const BlockArgs &a, cudaStream_t s) {
    cudaError_t e = launch_block<true, T>(p, a, s);
    if (e != cudaSuccess || p.cluster) return e;
    const int64_t G = a.rows / a.rows_per_gate;
    const int slices = block_slices(a.team || a.rows_per_gate == 1 ? 1 : G, a.D);
    // Few parts: 8 warps have them all in flight at once, and an SM holds the CTAs of
    // several blocks of columns (100 rows of D = 5248: 10.2 us; with 32 warps two
    // rounds of CTAs, 13).
    e = p.grid <= 8 * BR_BATCH && slices == 1 ? launch_block_reduce<T, 8>(p, a, slices, s)
                                              : launch_block_reduce<T, 32>(p, a, slices, s);
    if (e != cudaSuccess || slices == 1 || !a.w_post) return e;
    return launch_gw_reduce(a.part_post, a.gw_post, slices, a.D, s);
}

}  // namespace rmsn
