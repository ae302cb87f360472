// norm_q8.cuh -- kernels of the fused residual-add norm with an e4m3 output.
//
// HBM-bound: x and residual are read once, codes and new residual written once, a row's
// elements stay in registers between.  With v_j = h_j w'_j and a = max |v_j| over a group, the group's scale is r a / 448 and
// its codes are e4m3(v_j 448 / a): the norm's own factor r is the same for the whole row
// and cancels in the codes, so that the row's sum of squares and the groups' maxima come
// from one pass and cross the CTA through one barrier a row (groups of whole lanes need
// none for their codes).
//
//   Q8_STAGED  one row a CTA at a time out of a shared-memory ring that thread 0 fills
//              with 1-D bulk copies `stages` rows ahead; a stage is free again once every
//              thread has its units in registers, at the row's barrier.
//   Q8_DIRECT  one row a CTA from global memory: no more rows than CTAs fit at once.
//   Q8_WARP    short rows, one a warp, the next one's loads ahead of this one's sums.
//
// SHIFT: rows off 16-byte boundaries whose tensors all stand alike.  Units are then those
// of memory (hd columns in), the columns before and behind them one a thread; a CTA's rows
// all stand the same way.  A unit that crosses a group's border gives its first E - hd
// elements to the one group and the rest to the next, and the groups' maxima meet in
// shared memory.
#pragma once

#include "launch_util.h"
#include "norm_q8.h"
#include "quant.cuh"
#include "units.cuh"

namespace rmsn {

// The scale of a group and the factor of its codes.
__device__ __forceinline__ float2 q8_scale(uint32_t top, float r) {
    // (integers: NaN and infinity stay)
    const float a = __uint_as_float(max(top, __float_as_uint(least_top<RMSNORM_CACHE_E4M3>())));
    return make_float2(r * a * (1.f / 448.f), 448.f / a);
}

// The 8 (16-bit inputs) or 4 codes of a unit.
template <int E> __device__ __forceinline__ void store_codes(uint8_t *p, const float (&v)[E], float by, bool whole) {
    uint32_t c[E / 4];
#pragma unroll
    for (int i = 0; i < E / 4; ++i)
        c[i] = code_quad<RMSNORM_CACHE_E4M3>(v[4 * i] * by, v[4 * i + 1] * by, v[4 * i + 2] * by, v[4 * i + 3] * by);
    if (whole) {
        if constexpr (E == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(c[0], c[1]);
        else *reinterpret_cast<uint32_t *>(p) = c[0];
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) p[e] = (uint8_t)(c[e / 4] >> (8 * (e % 4)));
    }
}

// Maximum over aligned runs of n lanes (a power of two).
__device__ __forceinline__ uint32_t run_max(uint32_t v, int n) {
    for (int off = 1; off < n; off *= 2) v = max(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

template <typename T>
__device__ __forceinline__ void q8_issue(const Q8Args &a, uint64_t *full, unsigned char *data, int64_t row, int stage,
                                         uint64_t policy) {
    if (row == a.drop_row) return;
    const uint32_t bytes = (uint32_t)a.D * (uint32_t)sizeof(T);
    const uintptr_t px = (uintptr_t)(static_cast<const T *>(a.x) + row * a.ld_x);
    const uintptr_t pr = a.res ? (uintptr_t)(static_cast<const T *>(a.res) + row * a.ld_res) : 0;
    // the aligned superset of each row
    const uint32_t off = (uint32_t)(px & 15u), size = (off + bytes + 15u) & ~15u;  // (the tensors stand alike)
    unsigned char *dst = data + (size_t)stage * (a.res ? 2 : 1) * a.stage_bytes;
    mbar_arrive_expect_tx(&full[stage], a.res ? 2 * size : size);
    bulk_g2s(dst, reinterpret_cast<const void *>(px - off), size, &full[stage], policy);
    if (a.res) bulk_g2s(dst + a.stage_bytes, reinterpret_cast<const void *>(pr - off), size, &full[stage], policy);
}

// One row a CTA.  V units a thread.
template <typename T, bool RES, bool SHIFT, bool STAGED, int V, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) q8_row_kernel(const __grid_constant__ Q8Args a) {
    constexpr int E = vec_elems<T>(), MAXW = MAXT / 32;
    constexpr int MAXG = SHIFT ? MAXT * V * E / 32 + 2 : 1;  // groups of 32 columns
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float s_sum[2][MAXW];
    __shared__ uint32_t s_top[2][MAXW];
    __shared__ uint32_t s_group[SHIFT ? 3 : 1][MAXG];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, NT = blockDim.x, nw = NT >> 5;
    const int D = a.D;
    const float inv_D = 1.0f / (float)D;
    const bool grouped = a.group != 0;
    const int run = grouped ? a.group / E : 32;  // units (lanes) of a group
    const int64_t r0 = blockIdx.x, step = gridDim.x;
    // hd: columns before a row's first 16-byte boundary
    const int hd = SHIFT ? (int)(-((uintptr_t)(static_cast<const T *>(a.x) + r0 * a.ld_x)) & 15u) / (int)sizeof(T) : 0;
    const int NU = SHIFT ? min((D - hd) / E, V * NT) : D / E;
    const int cx = !SHIFT || t >= D - NU * E ? -1 : t < hd ? t : NU * E + t;  // this thread's single column

    uint64_t *full = reinterpret_cast<uint64_t *>(smem);
    unsigned char *data = smem + Q8_HEADER;
    uint64_t policy = 0;
    if constexpr (STAGED) {
        policy = l2_evict_first_policy();
        if (t == 0) {
            for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1);
            fence_mbar_init();
        }
    }
    if constexpr (SHIFT)
        for (int i = t; i < 3 * MAXG; i += NT) (&s_group[0][0])[i] = 0;
    if constexpr (STAGED || SHIFT) __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    if constexpr (STAGED)
        if (t == 0)
            for (int s = 0; s < a.stages && r0 + s * step < a.rows; ++s) q8_issue<T>(a, full, data, r0 + s * step, s, policy);

    uint4 vx[V], vr[RES ? V : 1], vw[V];
    float xx = 0.f, xr = 0.f, xw = 0.f;  // of column cx
    auto fetch = [&](const T *px, const T *pr) {  // at column hd
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = t + j * NT;
            if (u < NU) {
                vx[j] = STAGED ? reinterpret_cast<const uint4 *>(px)[u] : ld_stream(reinterpret_cast<const uint4 *>(px) + u);
                if constexpr (RES)
                    vr[j] = STAGED ? reinterpret_cast<const uint4 *>(pr)[u] : ld_stream(reinterpret_cast<const uint4 *>(pr) + u);
            }
        }
        if constexpr (SHIFT)
            if (cx >= 0) {
                xx = Cvt<T>::load1(px + (cx - hd));
                if constexpr (RES) xr = Cvt<T>::load1(pr + (cx - hd));
            }
    };
    auto fetch_global = [&](int64_t row) {
        fetch(static_cast<const T *>(a.x) + row * a.ld_x + hd,
              RES ? static_cast<const T *>(a.res) + row * a.ld_res + hd : nullptr);
    };
    if constexpr (!STAGED) fetch_global(r0);
    const T *wg = static_cast<const T *>(a.w);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int u = t + j * NT;
        if (u < NU) {
            if constexpr (SHIFT) {
                T c[E];
#pragma unroll
                for (int e = 0; e < E; ++e) c[e] = wg[hd + u * E + e];
                memcpy(&vw[j], c, 16);
            } else {
                vw[j] = __ldg(reinterpret_cast<const uint4 *>(wg) + u);
            }
        }
    }
    if constexpr (SHIFT)
        if (cx >= 0) xw = a.weight_bias + Cvt<T>::load1(wg + cx);

    int s = 0, buf = 0;
    uint32_t ph = 0;
    int64_t i = 0;
    for (int64_t row = r0; row < a.rows; row += step, ++i) {
        bool ok = true;
        if constexpr (STAGED) {
            const unsigned char *st = data + (size_t)s * (RES ? 2 : 1) * a.stage_bytes;
            const uint32_t off = SHIFT ? (uint32_t)((uintptr_t)(static_cast<const T *>(a.x) + row * a.ld_x) & 15u) : 0u;
            ok = mbar_wait_bounded(&full[s], ph, a.wait_budget);
            fetch(reinterpret_cast<const T *>(st + off) + hd, reinterpret_cast<const T *>(st + a.stage_bytes + off) + hd);
        }
        T *nres = RES ? static_cast<T *>(a.nres) + row * a.ld_nres + hd : nullptr;
        uint8_t *out = static_cast<uint8_t *>(a.out) + row * a.ld_out + hd;
        float v[V][E], ss = 0.f;
        uint32_t top = 0, part[V];  // part: a group's maximum so far
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = t + j * NT;
            part[j] = 0;
            if (u < NU) {
                float w[E];
                unpack_vec<T>(vx[j], v[j]);
                if constexpr (RES) {
                    float r[E];
                    unpack_vec<T>(vr[j], r);
#pragma unroll
                    for (int e = 0; e < E; ++e) v[j][e] += r[e];
                    if (ok) reinterpret_cast<uint4 *>(nres)[u] = pack_vec<T>(v[j]);
                }
                unpack_vec<T>(vw[j], w);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    ss = fmaf(v[j][e], v[j][e], ss);
                    v[j][e] *= a.weight_bias + w[e];
                }
                if constexpr (SHIFT) {
                    // a unit across a border: its first E - hd elements (all where hd = 0)
                    const int own = grouped && (u & (run - 1)) == run - 1 ? E - hd : E;
                    uint32_t next = 0;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        if (e < own) part[j] = max(part[j], magnitude(v[j][e]));
                        else next = max(next, magnitude(v[j][e]));
                    }
                    if (own < E) atomicMax(&s_group[buf][u / run + 1], next);
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e) part[j] = max(part[j], magnitude(v[j][e]));
                }
            }
        }
        float xv = 0.f;
        if constexpr (SHIFT)
            if (cx >= 0) {
                const float h = xx + xr;
                if constexpr (RES)
                    if (ok) Cvt<T>::store1(nres + (cx - hd), h);
                ss = fmaf(h, h, ss);
                xv = h * xw;
                if (grouped) atomicMax(&s_group[buf][cx >> a.group_shift], magnitude(xv));
                top = magnitude(xv);
            }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = t + j * NT;
            if (!grouped) {
                top = max(top, part[j]);
            } else {
                part[j] = run_max(part[j], run);
                if constexpr (SHIFT) {
                    if (u < NU && (u & (run - 1)) == 0) atomicMax(&s_group[buf][u / run], part[j]);
                } else if (ok && u < NU) {  // no need to wait for the row's sum
                    store_codes<E>(out + u * E, v[j], q8_scale(part[j], 1.f).y, a.whole_codes);
                }
            }
        }
        ss = group_sum<32>(ss);
        if (!grouped) top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) {
            s_sum[i & 1][warp] = ss;
            s_top[i & 1][warp] = top;
        }
        const bool bad = __syncthreads_or(!ok);
        if constexpr (STAGED) {
            if (bad) {  // leave once this CTA's copies have landed
                if (t == 0) {
                    atomicOr(a.status, DEVSTATUS_WAIT_TIMEOUT);
                    for (int64_t k = i; k < i + a.stages && r0 + k * step < a.rows; ++k)
                        if (r0 + k * step != a.drop_row)
                            mbar_wait_bounded(&full[k % a.stages], (uint32_t)((k / a.stages) & 1), DEFAULT_WAIT_BUDGET);
                }
                return;
            }
            if (t == 0 && row + a.stages * step < a.rows) q8_issue<T>(a, full, data, row + a.stages * step, s, policy);
        }
        ss = group_sum<32>(lane < nw ? s_sum[i & 1][lane] : 0.f);
        const float r = rsqrtf(ss * inv_D + a.eps);
        if (!grouped) {
            const float2 sc = q8_scale(__reduce_max_sync(0xffffffffu, lane < nw ? s_top[i & 1][lane] : 0u), r);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int u = t + j * NT;
                if (u < NU) store_codes<E>(out + u * E, v[j], sc.y, a.whole_codes);
            }
            if constexpr (SHIFT)
                if (cx >= 0) out[cx - hd] = (uint8_t)e4m3_pair(xv * sc.y, 0.f);
            if (t == 0) a.scale[row] = sc.x;
        } else if constexpr (SHIFT) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int u = t + j * NT;
                if (u < NU) {
                    const float by = q8_scale(s_group[buf][u / run], r).y;
                    if ((u & (run - 1)) == run - 1 && hd) {
                        const float next = q8_scale(s_group[buf][u / run + 1], r).y;
#pragma unroll
                        for (int e = 0; e < E; ++e) v[j][e] *= e < E - hd ? by : next;
                        store_codes<E>(out + u * E, v[j], 1.f, a.whole_codes);
                    } else {
                        store_codes<E>(out + u * E, v[j], by, a.whole_codes);
                    }
                }
            }
            if (cx >= 0) out[cx - hd] = (uint8_t)e4m3_pair(xv * q8_scale(s_group[buf][cx >> a.group_shift], r).y, 0.f);
            for (int g = t; g < a.groups; g += NT) {
                a.scale[row * a.groups + g] = q8_scale(s_group[buf][g], r).x;
            }
            // The buffer of two rows on was last read before this row's barrier, and is
            // next added to behind the next row's.
            const int far = buf == 0 ? 2 : buf - 1;
            for (int g = t; g <= a.groups; g += NT) s_group[far][g] = 0;
            buf = buf == 2 ? 0 : buf + 1;
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int u = t + j * NT;
                if (u < NU && (u & (run - 1)) == 0) a.scale[row * a.groups + u / run] = q8_scale(part[j], r).x;
            }
        }
        if constexpr (STAGED)
            if (++s == a.stages) {
                s = 0;
                ph ^= 1u;
            }
        if constexpr (!STAGED)
            if (row + step < a.rows) fetch_global(row + step);
    }
}

// One row a warp, V units a lane.
template <typename T, bool RES, int V>
__global__ void __launch_bounds__(Q8_WARP_NT, 2) q8_warp_kernel(const __grid_constant__ Q8Args a) {
    constexpr int E = vec_elems<T>();
    const int lane = threadIdx.x & 31, NU = a.D / E;
    const float inv_D = 1.0f / (float)a.D;
    const bool grouped = a.group != 0;
    const int run = grouped ? a.group / E : 32;
    const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
    griddep_wait();
    griddep_launch_dependents();
    uint4 vx[V], vr[RES ? V : 1], vw[V];
    auto fetch = [&](int64_t row) {
        const uint4 *px = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + row * a.ld_x);
        const uint4 *pr = RES ? reinterpret_cast<const uint4 *>(static_cast<const T *>(a.res) + row * a.ld_res) : nullptr;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = lane + 32 * j;
            if (u < NU) {
                vx[j] = ld_stream(px + u);
                if constexpr (RES) vr[j] = ld_stream(pr + u);
            }
        }
    };
    int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (row < a.rows) fetch(row);
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (lane + 32 * j < NU) vw[j] = __ldg(static_cast<const uint4 *>(a.w) + lane + 32 * j);
    for (; row < a.rows; row += step) {
        float v[V][E], ss = 0.f;
        uint32_t top = 0, part[V];
        uint4 *nres = RES ? reinterpret_cast<uint4 *>(static_cast<T *>(a.nres) + row * a.ld_nres) : nullptr;
        uint8_t *out = static_cast<uint8_t *>(a.out) + row * a.ld_out;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = lane + 32 * j;
            part[j] = 0;
            if (u < NU) {
                unpack_vec<T>(vx[j], v[j]);
                if constexpr (RES) {
                    float r[E];
                    unpack_vec<T>(vr[j], r);
#pragma unroll
                    for (int e = 0; e < E; ++e) v[j][e] += r[e];
                }
            }
        }
        // The next row may be this one's new residual's neighbour, never the same.
        if (row + step < a.rows) fetch(row + step);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = lane + 32 * j;
            if (u < NU) {
                float w[E];
                if constexpr (RES) nres[u] = pack_vec<T>(v[j]);
                unpack_vec<T>(vw[j], w);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    ss = fmaf(v[j][e], v[j][e], ss);
                    v[j][e] *= a.weight_bias + w[e];
                    part[j] = max(part[j], magnitude(v[j][e]));
                }
            }
            top = max(top, part[j]);
        }
        const float r = rsqrtf(group_sum<32>(ss) * inv_D + a.eps);
        const float2 whole = grouped ? make_float2(0.f, 0.f) : q8_scale(__reduce_max_sync(0xffffffffu, top), r);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = lane + 32 * j;
            const float2 sc = grouped ? q8_scale(run_max(part[j], run), r) : whole;
            if (u < NU) {
                store_codes<E>(out + u * E, v[j], sc.y, a.whole_codes);
                if (grouped && (u & (run - 1)) == 0) a.scale[row * a.groups + u / run] = sc.x;
            }
        }
        if (!grouped && lane == 0) a.scale[row] = whole.x;
    }
}

// Any row length, stride and alignment: one element a thread, the row read twice (the
// second time from L2).  Groups go to a warp each.
template <typename T, bool RES>
__global__ void __launch_bounds__(Q8_GENERIC_NT) q8_generic_kernel(const Q8Args a) {
    constexpr int NW = Q8_GENERIC_NT / 32;
    __shared__ float s_sum[NW];
    __shared__ uint32_t s_top[NW];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T *w = static_cast<const T *>(a.w);
    griddep_wait();
    griddep_launch_dependents();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + row * a.ld_x;
        const T *res = RES ? static_cast<const T *>(a.res) + row * a.ld_res : nullptr;
        auto h_of = [&](int j) { return RES ? Cvt<T>::load1(x + j) + Cvt<T>::load1(res + j) : Cvt<T>::load1(x + j); };
        auto weight = [&](int j) { return a.weight_bias + Cvt<T>::load1(w + j); };
        // a sum of sums of 64, so that rounding grows with neither length alone
        float ss = 0.f;
        uint32_t top = 0;
        for (int j0 = threadIdx.x; j0 < a.D; j0 += 64 * Q8_GENERIC_NT) {
            float part = 0.f;
            for (int i = 0, j = j0; i < 64 && j < a.D; ++i, j += Q8_GENERIC_NT) {
                const float h = h_of(j);
                part = fmaf(h, h, part);
                if (!a.group) top = max(top, magnitude(h * weight(j)));
            }
            ss += part;
        }
        ss = group_sum<32>(ss);
        top = __reduce_max_sync(0xffffffffu, top);
        __syncthreads();  // the row before has been read
        if (lane == 0) {
            s_sum[warp] = ss;
            s_top[warp] = top;
        }
        __syncthreads();
        ss = group_sum<32>(lane < NW ? s_sum[lane] : 0.f);
        const float r = rsqrtf(ss * (1.0f / (float)a.D) + a.eps);
        uint8_t *out = static_cast<uint8_t *>(a.out) + row * a.ld_out;
        T *nres = RES ? static_cast<T *>(a.nres) + row * a.ld_nres : nullptr;
        auto write = [&](int j, float h, float by) {
            out[j] = (uint8_t)e4m3_pair(h * weight(j) * by, 0.f);
            if (RES) Cvt<T>::store1(nres + j, h);
        };
        if (!a.group) {
            top = __reduce_max_sync(0xffffffffu, lane < NW ? s_top[lane] : 0u);
            const float2 s = q8_scale(top, r);
            for (int j = threadIdx.x; j < a.D; j += Q8_GENERIC_NT) write(j, h_of(j), s.y);
            if (threadIdx.x == 0) a.scale[row] = s.x;
        } else {
            for (int g = warp; g < a.groups; g += NW) {
                float h[4];
                uint32_t t = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = g * a.group + 32 * i + lane;
                    const bool in = 32 * i < a.group && j < a.D;
                    h[i] = in ? h_of(j) : 0.f;
                    if (in) t = max(t, magnitude(h[i] * weight(j)));
                }
                const float2 s = q8_scale(__reduce_max_sync(0xffffffffu, t), r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = g * a.group + 32 * i + lane;
                    if (32 * i < a.group && j < a.D) write(j, h[i], s.y);
                }
                if (lane == 0) a.scale[row * a.groups + g] = s.x;
            }
        }
    }
}

// Picks the instance for a plan.
template <typename T, bool RES, bool SHIFT, bool STAGED, int V, int MAXT, int MINB>
cudaError_t launch_q8_row(const Q8Plan &p, const Q8Args &a, cudaStream_t s) {
    static std::atomic<uint64_t> smem_mask{0};
    auto kern = q8_row_kernel<T, RES, SHIFT, STAGED, V, MAXT, MINB>;
    if (p.smem > 0) {
        const cudaError_t e = allow_max_dynamic_smem((const void *)kern, smem_mask);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kern, dim3(p.grid), dim3(p.threads), p.smem, s, a);
}

template <typename T, bool RES, bool SHIFT>
cudaError_t launch_q8_cta(const Q8Plan &p, const Q8Args &a, cudaStream_t s) {
    if (p.kind == Q8_DIRECT)
        return p.units == 1 ? launch_q8_row<T, RES, SHIFT, false, 1, 512, 2>(p, a, s)
                            : launch_q8_row<T, RES, SHIFT, false, 2, 1024, 1>(p, a, s);
    if (p.threads <= 256) return launch_q8_row<T, RES, SHIFT, true, 2, 256, 4>(p, a, s);
    if (p.threads <= 512) return launch_q8_row<T, RES, SHIFT, true, 2, 512, 2>(p, a, s);
    return launch_q8_row<T, RES, SHIFT, true, 2, 1024, 1>(p, a, s);
}

template <typename T, bool RES> cudaError_t launch_q8_kind(const Q8Plan &p, const Q8Args &a, cudaStream_t s) {
    if (p.kind == Q8_GENERIC) return launch_pdl(q8_generic_kernel<T, RES>, dim3(p.grid), dim3(p.threads), 0, s, a);
    if (p.kind == Q8_WARP)
        return launch_pdl(p.units == 1   ? q8_warp_kernel<T, RES, 1>
                          : p.units == 2 ? q8_warp_kernel<T, RES, 2>
                                         : q8_warp_kernel<T, RES, 4>,
                          dim3(p.grid), dim3(p.threads), 0, s, a);
    return p.shift ? launch_q8_cta<T, RES, true>(p, a, s) : launch_q8_cta<T, RES, false>(p, a, s);
}

template <typename T> cudaError_t launch_q8_any(const Q8Plan &p, const Q8Args &a, cudaStream_t s) {
    if (!q8_plan_ok(p)) return cudaErrorInvalidConfiguration;
    return a.res ? launch_q8_kind<T, true>(p, a, s) : launch_q8_kind<T, false>(p, a, s);
}

}  // namespace rmsn
