// block_generic.cuh -- the norm pair around a block for any row length and
// alignment, and the second stage of its weight and gate gradients.
//
// One CTA per row at a time, one unit (16 bytes, or an element off 16-byte
// boundaries) per thread and step; a row is read from global memory or L2 once per
// pass (forward: sum of y^2, sum of h^2, outputs), and the VJP's sums are kept in
// its scratch.  It takes the rows the tiers that hold a row on chip cannot: 2000 of D =
// 20000 (bf16) forward in 75 us, 64 % of the copy bandwidth (198 an element at a
// time), VJP in 253 us, 28 % (465): its sums are read and written for every row.
#pragma once

#include "block.h"
#include "units.cuh"

namespace rmsn {

constexpr int BLOCK_GENERIC_NT = 512;

// Sum of v over the CTA, the same in every thread: warp butterfly, then the
// warp totals in warp order.  `red` holds a float a warp; the CTA passes two
// barriers.
template <int NT>
__device__ __forceinline__ float cta_sum(float v, float *red) {
    v = group_sum<32>(v);
    __syncthreads();  // the previous sum has been read
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) t += red[w];
    return t;
}

// A row's units of UB bytes: E elements of unit u, and those of an fp32 row.
template <typename T, int UB> struct GenericUnit {
    static constexpr int E = UB / (int)sizeof(T);
    using Unit = typename RawUnit<UB>::type;
    static __device__ __forceinline__ void load(const void *row, int u, float (&f)[E]) {
        unpack_unit<T, UB>(static_cast<const Unit *>(row)[u], f);
    }
    static __device__ __forceinline__ void store(void *row, int u, const float (&f)[E]) {
        static_cast<Unit *>(row)[u] = pack_unit<T, UB>(f);
    }
    static __device__ __forceinline__ void load_floats(const float *row, int u, float (&f)[E]) {
        if constexpr (E >= 4) {
#pragma unroll
            for (int k = 0; k < E / 4; ++k) {
                const float4 v = reinterpret_cast<const float4 *>(row)[u * (E / 4) + k];
                f[4 * k] = v.x;
                f[4 * k + 1] = v.y;
                f[4 * k + 2] = v.z;
                f[4 * k + 3] = v.w;
            }
        } else {
            f[0] = row[u];
        }
    }
    static __device__ __forceinline__ void store_floats(float *row, int u, const float (&f)[E]) {
        if constexpr (E >= 4) {
#pragma unroll
            for (int k = 0; k < E / 4; ++k)
                reinterpret_cast<float4 *>(row)[u * (E / 4) + k] =
                    make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
        } else {
            row[u] = f[0];
        }
    }
};

template <typename T, int UB>
__global__ void __launch_bounds__(BLOCK_GENERIC_NT, 3) block_fwd_generic_kernel(const BlockArgs a) {
    using GU = GenericUnit<T, UB>;
    constexpr int NT = BLOCK_GENERIC_NT, E = GU::E;
    __shared__ float red[NT / 32];
    const int tid = threadIdx.x, NU = a.D / E;
    const float wb = a.weight_bias, inv_D = 1.0f / (float)a.D;
    griddep_wait();
    griddep_launch_dependents();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *y = static_cast<const T *>(a.y) + row * a.ld_y;
        const T *res = static_cast<const T *>(a.res) + row * a.ld_res;
        const T *gate = a.gate ? static_cast<const T *>(a.gate) + gate_row(row, a.rows_per_gate) * a.ld_gate : nullptr;
        T *out = static_cast<T *>(a.out0) + row * a.ld_out0;
        T *nres = static_cast<T *>(a.out1) + row * a.ld_out1;
        float r_y = 1.f;
        if (a.w_post) {
            float s = 0.f;
            for (int u = tid; u < NU; u += NT) {
                float v[E];
                GU::load(y, u, v);
#pragma unroll
                for (int e = 0; e < E; ++e) s = fmaf(v[e], v[e], s);
            }
            r_y = rsqrtf(cta_sum<NT>(s, red) * inv_D + a.eps);
        }
        auto joined = [&](int u, float (&h)[E]) {
            float m[E], x[E];
            GU::load(y, u, m);
#pragma unroll
            for (int e = 0; e < E; ++e) m[e] *= a.scale * r_y;
            if (gate) {
                GU::load(gate, u, x);
#pragma unroll
                for (int e = 0; e < E; ++e) m[e] *= x[e];
            }
            if (a.w_post) {
                GU::load(a.w_post, u, x);
#pragma unroll
                for (int e = 0; e < E; ++e) m[e] *= wb + x[e];
            }
            GU::load(res, u, h);
#pragma unroll
            for (int e = 0; e < E; ++e) h[e] += m[e];
        };
        float s = 0.f;
        for (int u = tid; u < NU; u += NT) {
            float h[E];
            joined(u, h);
#pragma unroll
            for (int e = 0; e < E; ++e) s = fmaf(h[e], h[e], s);
        }
        const float r_h = rsqrtf(cta_sum<NT>(s, red) * inv_D + a.eps);
        for (int u = tid; u < NU; u += NT) {
            float h[E], w[E];
            joined(u, h);
            GU::load(a.w_pre, u, w);
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] = h[e] * r_h * (wb + w[e]);
            GU::store(nres, u, h);
            GU::store(out, u, w);
        }
        if (a.rstd && tid == 0) {
            a.rstd[row] = r_y;
            a.rstd[a.rows + row] = r_h;
        }
    }
}

template <typename T, int UB>
__global__ void __launch_bounds__(BLOCK_GENERIC_NT, 2) block_vjp_generic_kernel(const BlockArgs a) {
    using GU = GenericUnit<T, UB>;
    constexpr int NT = BLOCK_GENERIC_NT, E = GU::E;
    __shared__ float red[NT / 32];
    const int tid = threadIdx.x, D = a.D, NU = D / E;
    const float wb = a.weight_bias, inv_D = 1.0f / (float)D;
    const bool post = a.w_post != nullptr;
    const int64_t cta = blockIdx.x;
    const int64_t r0 = split_first(cta, a.split_q, a.split_r), r1 = split_first(cta + 1, a.split_q, a.split_r);
    const bool per_row = a.gate && a.rows_per_gate == 1;
    griddep_wait();
    griddep_launch_dependents();
    float *pre = a.part_pre + cta * D;
    for (int64_t row = r0; row < r1; ++row) {
        const int64_t gr = gate_row(row, a.rows_per_gate);
        const T *y = static_cast<const T *>(a.y) + row * a.ld_y;
        const T *hp = static_cast<const T *>(a.res) + row * a.ld_res;
        const T *g = static_cast<const T *>(a.g) + row * a.ld_g;
        const T *gres = a.g_res ? static_cast<const T *>(a.g_res) + row * a.ld_g_res : nullptr;
        const T *gate = a.gate ? static_cast<const T *>(a.gate) + gr * a.ld_gate : nullptr;
        T *gy = static_cast<T *>(a.out0) + row * a.ld_out0;
        T *gh = static_cast<T *>(a.out1) + row * a.ld_out1;
        float r_y = 1.f, r_h;
        if (a.rstd) {
            if (post) r_y = a.rstd[row];
            r_h = a.rstd[a.rows + row];
        } else {
            float sy = 0.f, sh = 0.f;
            for (int u = tid; u < NU; u += NT) {
                float v[E], h[E];
                GU::load(y, u, v);
                GU::load(hp, u, h);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    sy = fmaf(v[e], v[e], sy);
                    sh = fmaf(h[e], h[e], sh);
                }
            }
            if (post) r_y = rsqrtf(cta_sum<NT>(sy, red) * inv_D + a.eps);
            r_h = rsqrtf(cta_sum<NT>(sh, red) * inv_D + a.eps);
        }
        float s = 0.f;
        for (int u = tid; u < NU; u += NT) {
            float x[E], w[E], h[E];
            GU::load(g, u, x);
            GU::load(a.w_pre, u, w);
            GU::load(hp, u, h);
#pragma unroll
            for (int e = 0; e < E; ++e) s = fmaf(x[e] * (wb + w[e]), h[e], s);
        }
        const float cc = r_h * (r_h * (cta_sum<NT>(s, red) * inv_D));  // r_h^2 alone can leave fp32's range
        // g_h, with g and h of the unit
        auto grad_h = [&](int u, float (&v)[E], float (&x)[E], float (&h)[E]) {
            float w[E];
            GU::load(g, u, x);
            GU::load(a.w_pre, u, w);
            GU::load(hp, u, h);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = r_h * (x[e] * (wb + w[e]) - h[e] * cc);
            if (gres) {
                GU::load(gres, u, w);
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] += w[e];
            }
        };
        auto mult = [&](int u, float (&m)[E]) {
            float x[E];
#pragma unroll
            for (int e = 0; e < E; ++e) m[e] = a.scale;
            if (gate) {
                GU::load(gate, u, x);
#pragma unroll
                for (int e = 0; e < E; ++e) m[e] *= x[e];
            }
            if (post) {
                GU::load(a.w_post, u, x);
#pragma unroll
                for (int e = 0; e < E; ++e) m[e] *= wb + x[e];
            }
        };
        float ee = 0.f;
        if (post) {
            s = 0.f;
            for (int u = tid; u < NU; u += NT) {
                float v[E], x[E], h[E], m[E], yv[E];
                grad_h(u, v, x, h);
                mult(u, m);
                GU::load(y, u, yv);
#pragma unroll
                for (int e = 0; e < E; ++e) s = fmaf(m[e] * v[e], yv[e], s);
            }
            ee = r_y * (r_y * (cta_sum<NT>(s, red) * inv_D));
        }
        // this gate row's sum: whole here (its own row of g_gate), or a part
        const bool whole = a.g_gate && gr * a.rows_per_gate >= r0 && (gr + 1) * a.rows_per_gate <= r1;
        float *mid = per_row ? a.part_mid + 2 * cta * D
                     : whole ? a.g_gate + gr * D
                             : a.part_mid + mid_slot(cta, gr == gate_row(r0, a.rows_per_gate)) * D;
        const bool first = per_row ? row == r0 : row == r0 || row % a.rows_per_gate == 0;
        for (int u = tid; u < NU; u += NT) {
            float v[E], x[E], h[E], m[E], yv[E], sum[E], q[E];
            grad_h(u, v, x, h);
            mult(u, m);
            GU::load(y, u, yv);
            if (row != r0) GU::load_floats(pre, u, sum);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float p = x[e] * h[e] * r_h;
                sum[e] = row == r0 ? p : sum[e] + p;
                q[e] = a.scale * v[e] * yv[e] * r_y;
            }
            GU::store_floats(pre, u, sum);
            if (per_row) {
                float w[E];
                if (post) GU::load(a.w_post, u, w);
#pragma unroll
                for (int e = 0; e < E; ++e) w[e] = post ? q[e] * (wb + w[e]) : q[e];
                GU::store_floats(a.g_gate + gr * D, u, w);
                GU::load(gate, u, w);
#pragma unroll
                for (int e = 0; e < E; ++e) q[e] *= w[e];
            }
            if (!first) {
                GU::load_floats(mid, u, sum);
#pragma unroll
                for (int e = 0; e < E; ++e) q[e] += sum[e];
            }
            GU::store_floats(mid, u, q);
            GU::store(gh, u, v);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = r_y * (m[e] * v[e] - yv[e] * ee);
            GU::store(gy, u, v);
        }
    }
}

// Second stage: a CTA covers 32 columns with W warps.
//   gw_pre = the CTAs' partial rows, each warp a contiguous run of them, the
//   warps' sums added in warp order.
//   A of each gate row: with fewer gate rows than warps, W / G warps share a gate
//   row's parts; with more, warp k takes the gate rows k, k + W, ...  A part is a row of part_mid, or the whole sum that one CTA
//   left in g_gate, which becomes w2 * A in place.  Gate rows of one row each
//   come finished from the first stage, which also weighted its sums.
// With many gate rows the grid has slices in y, each with a run of them, whose
// sums of gw_post the library's column sum then adds.
// The order of every sum depends on how the rows are dealt out alone.  Latency-bound: a
// warp's first loads of both sums are in flight together, and the row
// arithmetic is 32-bit (I) where the row count allows (64-bit divisions made
// the whole stage 14 us at 16384 x 4096 in 8 gate rows).
constexpr int BR_BATCH = 16;

template <typename T, typename I, int W>
__global__ void __launch_bounds__(32 * W) block_reduce_kernel(const BlockArgs a, int grid) {
    __shared__ float sums[2][W][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = a.D;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    const bool in = col < D;
    const T *w2 = static_cast<const T *>(a.w_post);
    const T *gate = static_cast<const T *>(a.gate);
    const I rows = (I)a.rows, rpg = (I)a.rows_per_gate, G = rows / rpg;
    const I q = (I)a.split_q, r = (I)a.split_r;
    const bool need_mid = w2 || gate, per_row = gate && rpg == 1;
    const int team = G >= W ? 1 : W / (int)G;  // warps a gate row
    const int per = (grid + W - 1) / W;
    const int p0 = min(grid, warp * per), p1 = min(grid, p0 + per);
    // CTAs c0 .. c1 have gate row gr's rows (as vjp_rows deals them out); the warps
    // of a team take equal runs of them
    auto ctas_of = [&](I gr, I &c0, I &c1) {
        if (a.team) {
            c0 = (I)split_first(gr, q, r);
            c1 = (I)split_first((int64_t)gr + 1, q, r) - 1;
        } else {
            c0 = split_part<I>(gr * rpg, q, r);
            c1 = split_part<I>(gr * rpg + (rpg - 1), q, r);
        }
    };
    // c0's part of gr is its second one unless gr is its first gate row
    auto slot_of = [&](I c0, I gr) {
        return mid_slot(c0, a.team || (I)split_first(c0, q, r) / rpg == gr);
    };
    // Up to BR_BATCH of n rows of a [*, D] array, `step` rows apart from p on, at this column.
    auto load_rows = [&](const float *p, int64_t step, int n, float (&v)[BR_BATCH]) {
#pragma unroll
        for (int i = 0; i < BR_BATCH; ++i) {
            v[i] = i < n ? *p : 0.f;
            p += step;
        }
    };
    // s plus n rows from p on in order, the first of them in v already
    auto add_rows = [&](const float *p, int64_t step, int n, float (&v)[BR_BATCH], float s) {
        while (true) {
#pragma unroll
            for (int i = 0; i < BR_BATCH; ++i) s += v[i];
            n -= BR_BATCH;
            if (n <= 0) return s;
            p += BR_BATCH * step;
            load_rows(p, step, n, v);
        }
    };
    griddep_wait();
    griddep_launch_dependents();
    const bool pre_here = blockIdx.y == 0;  // the slices share out the gate rows alone
    const int pre_n = in && pre_here ? p1 - p0 : 0;
    const float *pre_p = a.part_pre + (int64_t)p0 * D + col;
    float head[BR_BATCH];
    load_rows(pre_p, D, pre_n, head);  // in flight while the gate rows are found
    const float w2c = in && w2 ? a.weight_bias + Cvt<T>::load1(w2 + col) : 1.f;
    float post = 0.f, gt = 1.f;
    if (need_mid && per_row) {
        const float *p = a.part_mid + 2 * (int64_t)p0 * D + col;
        float v[BR_BATCH];
        load_rows(p, 2 * (int64_t)D, in ? p1 - p0 : 0, v);
        post = add_rows(p, 2 * (int64_t)D, in ? p1 - p0 : 0, v, 0.f);
    } else if (need_mid) {
        const int mate = warp % team;
        const I g0 = (I)((uint64_t)G * blockIdx.y / gridDim.y), g1 = (I)((uint64_t)G * (blockIdx.y + 1) / gridDim.y);
        for (I gr = g0 + warp / team; gr < g1; gr += W / team) {
            I c0, c1;
            ctas_of(gr, c0, c1);
            float A = 0.f;
            if (in && gate && mate == 0) gt = Cvt<T>::load1(gate + (int64_t)gr * a.ld_gate + col);
            if (c0 == c1 && a.g_gate) {
                if (mate == 0 && in) A = a.g_gate[(int64_t)gr * D + col];
            } else {
                // parts: CTA c0's, then c0 + 1 ... c1 (each its first gate row)
                const int n = (int)(c1 - c0) + 1, share = (n + team - 1) / team;
                int i0 = min(n, mate * share);
                const int i1 = min(n, i0 + share);
                const float *first = nullptr;
                if (i0 == 0 && i1 > 0) {
                    first = a.part_mid + slot_of(c0, gr) * D + col;
                    i0 = 1;
                }
                const int more = in ? i1 - i0 : 0;
                const float *p = a.part_mid + 2 * ((int64_t)c0 + i0) * D + col;
                float v[BR_BATCH];
                load_rows(p, 2 * (int64_t)D, more, v);
                if (first && in) A = *first;
                A = add_rows(p, 2 * (int64_t)D, more, v, A);
            }
            if (team == 1 && in) {
                if (gate) a.g_gate[(int64_t)gr * D + col] = A * w2c;
                post = fmaf(gt, A, post);
            }
            if (team > 1) post = A;  // this warp's part of its gate row's A
        }
    }
    sums[0][warp][lane] = add_rows(pre_p, D, pre_n, head, 0.f);
    sums[1][warp][lane] = post;
    __syncthreads();
    if (warp == 0 && in && pre_here) {
        float t = sums[0][0][lane];
#pragma unroll
        for (int k = 1; k < W; ++k) t += sums[0][k][lane];
        a.gw_pre[col] = t;
    }
    if (!need_mid) return;
    const int places = per_row || team == 1 ? W : (int)G;  // what gw_post adds up
    if (places == (int)G && team > 1) {  // each team's first warp joins its gate row's parts
        float A = 0.f;
        if (warp % team == 0 && warp / team < (int)G) {
            for (int k = 0; k < team; ++k) A += sums[1][warp + k][lane];
            if (gate && in) a.g_gate[(int64_t)(warp / team) * D + col] = A * w2c;
        }
        __syncthreads();
        if (warp % team == 0 && warp / team < (int)G) sums[1][warp / team][lane] = gt * A;
        __syncthreads();
    }
    if (warp == 1 && in && w2) {
        float t = 0.f;
        for (int k = 0; k < places; ++k) t += sums[1][k][lane];
        (gridDim.y == 1 ? a.gw_post : a.part_post + (size_t)blockIdx.y * D)[col] = t;
    }
}

}  // namespace rmsn
