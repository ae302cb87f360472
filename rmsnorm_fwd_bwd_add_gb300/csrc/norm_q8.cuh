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
//   Q8_LONG, Q8_GENERIC  rows that do not fit, or whose tensors stand differently to
//              16-byte boundaries, read twice.
//
// SHIFT: rows off 16-byte boundaries whose tensors all stand alike.  Units are then those
// of memory (hd columns in), the columns before and behind them one a thread; a CTA's rows
// all stand the same way.  A unit that crosses a group's border gives its first E - hd
// elements to the one group and the rest to the next, and the groups' maxima meet in
// shared memory.
//
// On the GB300 (6.8 TB/s copied), inputs changing from call to call: 16384 x 8192 bf16 with
// residual 147 us (94 % of that), 8192 x 12288 in groups of 128 109 us (96 %), 16384 x 4096
// 73 us (95 %); without a residual 8192 x 4096 fp16 in groups of 128 21 us (72 %: 3 bytes an
// element for the same instructions, whose latency the 16 warps that fit an SM at 106
// registers, 32 of them the weights, do not cover: 57 % of the issue slots used); off 16-byte
// boundaries 16384 x 4097 78 us (88 %), 5000 x 4097 in groups 30 us (71 %: the same, unaligned
// weights at the start, 8.2 rows a CTA); 4 x 4096 2.2 us.
#pragma once

#include "launch_util.h"
#include "norm_q8.h"
#include "quant.cuh"
#include "units.cuh"

namespace rmsn {

// The scale of a group and the factor of its codes, its first part alone: v is rounded before
// it, so that few quotients are borders of codes still (5000 x 4097 with residual in groups
// of 128: of 41 million codes 245 are not those of 64 bits, 366 in the plain form in fp32,
// 185 with both parts, which take 33.4 us where this takes 30.0, and 8192 x 4096 without
// residual 22.0 where this takes 21.0).
__device__ __forceinline__ float2 q8_scale(float top, float r) {
    const float a = scaled_top<RMSNORM_CACHE_E4M3>(top);
    return make_float2(r * a * (1.f / 448.f), code_factor<RMSNORM_CACHE_E4M3>(a).x);
}

// The 8 (16-bit inputs) or 4 codes of a unit, P pairs of values, stored if `in`.
template <int P> __device__ __forceinline__ void store_codes(uint8_t *p, const float2 (&v)[P], float by, bool whole, bool in) {
    uint32_t c[P / 2];
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
        const float2 a = f2mul(v[2 * i], make_float2(by, by)), b = f2mul(v[2 * i + 1], make_float2(by, by));
        c[i] = code_quad<RMSNORM_CACHE_E4M3>(a.x, a.y, b.x, b.y);
    }
    if (whole) {
        if constexpr (P == 4) {
            if (in) *reinterpret_cast<uint2 *>(p) = make_uint2(c[0], c[1]);
        } else {
            if (in) *reinterpret_cast<uint32_t *>(p) = c[0];
        }
    } else if (in) {
#pragma unroll
        for (int e = 0; e < 2 * P; ++e) p[e] = (uint8_t)(c[e / 4] >> (8 * (e % 4)));
    }
}

// run_max of V values at once.  Runs of 16 lanes (128 columns of 16 bits) are unrolled: 8192
// rows of fp16, D = 4096 take 22.4 us with the loop, 20.9 so, and 25.6 with reductions of a
// part of the warp's lanes in one instruction.  Runs of 8 unrolled as well gain in their own
// groups and lose in others (these rows in groups of 64 21.3 -> 20.7 us, 128 20.9 -> 21.0; fp32
// 16384 x 2048 in groups of 32 40.2 -> 38.6, 64 39.7 -> 39.9, 128 37.0 -> 37.3), runs of 4 too
// lose (fp16 in groups of 32 20.9 -> 21.3, 64 21.6, 128 22.1).
template <int V> __device__ __forceinline__ void run_maxima(float (&top)[V], int n) {
    auto step = [&](int off) {
#pragma unroll
        for (int j = 0; j < V; ++j) top[j] = max_abs(top[j], __shfl_xor_sync(0xffffffffu, top[j], off));
    };
    if (n == 32) {
#pragma unroll
        for (int j = 0; j < V; ++j) top[j] = warp_max(top[j]);
    } else if (n == 16) {
#pragma unroll
        for (int off = 1; off < 16; off *= 2) step(off);
    } else {
        for (int off = 1; off < n; off *= 2) step(off);
    }
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
    constexpr int E = vec_elems<T>(), P = vec_pairs<T>(), MAXW = MAXT / 32;
    constexpr int MAXG = SHIFT ? MAXT * V * E / 32 + 2 : 1;  // groups of 32 columns
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float2 s_row[2][MAXW];  // a warp's sum of squares and largest value
    __shared__ uint32_t s_group[SHIFT ? 3 : 1][MAXG];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, NT = blockDim.x, nw = NT >> 5;
    const int D = a.D;
    const float inv_D = 1.0f / (float)D;
    const bool grouped = a.group != 0;
    const int run = grouped ? a.group / E : 32, run_shift = 31 - __clz(run);  // units (lanes) of a group
    const int64_t r0 = blockIdx.x, step = gridDim.x;
    // hd: columns before a row's first 16-byte boundary
    const int hd = SHIFT ? (int)(-((uintptr_t)(static_cast<const T *>(a.x) + r0 * a.ld_x)) & 15u) / (int)sizeof(T) : 0;
    const int NU = SHIFT ? min((D - hd) / E, V * NT) : D / E;
    const int cx = !SHIFT || t >= D - NU * E ? -1 : t < hd ? t : NU * E + t;  // this thread's single column
    // SHIFT: whether this thread's units cross a group's border, their first E - hd elements
    // before it (a CTA's threads are whole groups)
    const bool crosses = SHIFT && grouped && hd && (t & (run - 1)) == run - 1;

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

    // A thread's units past the row are zeros, and its loops run over all V of them: with a
    // branch around each, none of their work overlapped.
    uint4 vx[V], vr[RES ? V : 1];
    float xx = 0.f, xr = 0.f, xw = 0.f;  // of column cx
    auto fetch = [&](const T *px, const T *pr) {  // at column hd
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = t + j * NT;
            vx[j] = make_uint4(0, 0, 0, 0);
            if constexpr (RES) vr[j] = make_uint4(0, 0, 0, 0);
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
    if constexpr (!STAGED)
        fetch(static_cast<const T *>(a.x) + r0 * a.ld_x + hd, RES ? static_cast<const T *>(a.res) + r0 * a.ld_res + hd : nullptr);
    const T *wg = static_cast<const T *>(a.w);
    float2 w[V][P];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int u = t + j * NT;
        uint4 c = make_uint4(0, 0, 0, 0);
        if (u < NU) {
            if constexpr (SHIFT) {
                T e1[E];
#pragma unroll
                for (int e = 0; e < E; ++e) e1[e] = wg[hd + u * E + e];
                memcpy(&c, e1, 16);
            } else {
                c = __ldg(reinterpret_cast<const uint4 *>(wg) + u);
            }
        }
        unpack_vec<T>(c, w[j]);
#pragma unroll
        for (int m = 0; m < P; ++m) w[j][m] = f2add(w[j][m], make_float2(a.weight_bias, a.weight_bias));
    }
    if constexpr (SHIFT)
        if (cx >= 0) xw = a.weight_bias + Cvt<T>::load1(wg + cx);

    int s = 0, buf = 0, side = 0;
    uint32_t ph = 0;
    for (int64_t row = r0; row < a.rows; row += step) {
        bool ok = true;
        if constexpr (STAGED) {
            const unsigned char *st = data + (size_t)s * (RES ? 2 : 1) * a.stage_bytes;
            const uint32_t off = SHIFT ? (uint32_t)((uintptr_t)(static_cast<const T *>(a.x) + row * a.ld_x) & 15u) : 0u;
            ok = mbar_wait_bounded(&full[s], ph, a.wait_budget);
            fetch(reinterpret_cast<const T *>(st + off) + hd, reinterpret_cast<const T *>(st + a.stage_bytes + off) + hd);
        }
        T *nres = RES ? static_cast<T *>(a.nres) + row * a.ld_nres + hd : nullptr;
        uint8_t *out = static_cast<uint8_t *>(a.out) + row * a.ld_out + hd;
        float2 v[V][P], s2 = make_float2(0.f, 0.f);
        float part[V];  // a unit's largest value
#pragma unroll
        for (int j = 0; j < V; ++j) {
            unpack_vec<T>(vx[j], v[j]);
            if constexpr (RES) {
                float2 r[P];
                unpack_vec<T>(vr[j], r);
#pragma unroll
                for (int m = 0; m < P; ++m) v[j][m] = f2add(v[j][m], r[m]);
                if (ok && t + j * NT < NU) reinterpret_cast<uint4 *>(nres)[t + j * NT] = pack_vec<T>(v[j]);
            }
            part[j] = 0.f;
#pragma unroll
            for (int m = 0; m < P; ++m) {
                s2 = f2fma(v[j][m], v[j][m], s2);
                v[j][m] = f2mul(v[j][m], w[j][m]);
                part[j] = max_abs(part[j], v[j][m].x, v[j][m].y);
            }
        }
        if constexpr (SHIFT)
            if (crosses) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float next = 0.f;
                    part[j] = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float x = e & 1 ? v[j][e / 2].y : v[j][e / 2].x;
                        if (e < E - hd) part[j] = max_abs(part[j], x);
                        else next = max_abs(next, x);
                    }
                    if (t + j * NT < NU) atomicMax(&s_group[buf][((t + j * NT) >> run_shift) + 1], __float_as_uint(next));
                }
            }
        float xv = 0.f, ss = s2.x + s2.y, top = 0.f;
        if constexpr (SHIFT)
            if (cx >= 0) {
                const float h = xx + xr;
                if constexpr (RES)
                    if (ok) Cvt<T>::store1(nres + (cx - hd), h);
                ss = fmaf(h, h, ss);
                xv = h * xw;
                if (grouped) atomicMax(&s_group[buf][cx >> a.group_shift], __float_as_uint(max_abs(0.f, xv)));
                top = max_abs(0.f, xv);
            }
        if (grouped) {
            run_maxima(part, run);
            if constexpr (SHIFT) {
                if ((t & (run - 1)) == 0) {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (t + j * NT < NU) atomicMax(&s_group[buf][(t + j * NT) >> run_shift], __float_as_uint(part[j]));
                }
            } else if (ok) {  // no need to wait for the row's sum
#pragma unroll
                for (int j = 0; j < V; ++j)
                    store_codes(out + (t + j * NT) * E, v[j], q8_scale(part[j], 1.f).y, a.whole_codes, t + j * NT < NU);
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) top = max_abs(top, part[j]);
            top = warp_max(top);
        }
        ss = group_sum<32>(ss);
        if (lane == 0) s_row[side][warp] = make_float2(ss, top);
        const bool bad = __syncthreads_or(!ok);
        if constexpr (STAGED) {
            if (bad) {  // leave once this CTA's copies have landed
                if (t == 0) {
                    atomicOr(a.status, DEVSTATUS_WAIT_TIMEOUT);
                    const int64_t i = (row - r0) / step;
                    for (int64_t k = i; k < i + a.stages && r0 + k * step < a.rows; ++k)
                        if (r0 + k * step != a.drop_row)
                            mbar_wait_bounded(&full[k % a.stages], (uint32_t)((k / a.stages) & 1), DEFAULT_WAIT_BUDGET);
                }
                return;
            }
            if (t == 0 && row + a.stages * step < a.rows) q8_issue<T>(a, full, data, row + a.stages * step, s, policy);
        }
        // every lane of MAXW has a warp's, the next MAXW lanes the same again
        const float2 mine = (lane & (MAXW - 1)) < nw ? s_row[side][lane & (MAXW - 1)] : make_float2(0.f, 0.f);
        side ^= 1;
        const float r = rsqrtf(group_sum<MAXW>(mine.x) * inv_D + a.eps);
        if (!grouped) {
            const float2 sc = q8_scale(run_max(mine.y, MAXW), r);
#pragma unroll
            for (int j = 0; j < V; ++j) store_codes(out + (t + j * NT) * E, v[j], sc.y, a.whole_codes, t + j * NT < NU);
            if constexpr (SHIFT)
                if (cx >= 0) out[cx - hd] = (uint8_t)e4m3_pair(xv * sc.y, 0.f);
            if (t == 0) a.scale[row] = sc.x;
        } else if constexpr (SHIFT) {
            auto scale_of = [&](int g) { return q8_scale(__uint_as_float(s_group[buf][g]), r); };
            float by[V];
#pragma unroll
            for (int j = 0; j < V; ++j) by[j] = t + j * NT < NU ? scale_of((t + j * NT) >> run_shift).y : 0.f;
            if (crosses) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (t + j * NT < NU) {
                        const float next = scale_of(((t + j * NT) >> run_shift) + 1).y;
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            float &x = e & 1 ? v[j][e / 2].y : v[j][e / 2].x;
                            x *= e < E - hd ? by[j] : next;
                        }
                        by[j] = 1.f;
                    }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) store_codes(out + (t + j * NT) * E, v[j], by[j], a.whole_codes, t + j * NT < NU);
            if (cx >= 0) out[cx - hd] = (uint8_t)e4m3_pair(xv * scale_of(cx >> a.group_shift).y, 0.f);
            for (int g = t; g < a.groups; g += NT) a.scale[row * a.groups + g] = scale_of(g).x;
            // The buffer of two rows on was last read before this row's barrier, and is
            // next added to behind the next row's.
            const int far = buf == 0 ? 2 : buf - 1;
            for (int g = t; g <= a.groups; g += NT) s_group[far][g] = 0;
            buf = buf == 2 ? 0 : buf + 1;
        } else if ((t & (run - 1)) == 0) {
            float *scale = a.scale + row * a.groups;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (t + j * NT < NU) scale[(t + j * NT) >> run_shift] = q8_scale(part[j], r).x;
        }
        if constexpr (STAGED)
            if (++s == a.stages) {
                s = 0;
                ph ^= 1u;
            }
    }
}

// One row a warp, V units a lane (16384 x 1024 bf16 21 us, 83 %; 16384 x 512 fp16 in groups of
// 64 12 us, 72 %: a row's trip to memory for each of a warp's few rows).
template <typename T, bool RES, int V>
__global__ void __launch_bounds__(Q8_WARP_NT, 2) q8_warp_kernel(const __grid_constant__ Q8Args a) {
    constexpr int E = vec_elems<T>(), P = vec_pairs<T>();
    const int lane = threadIdx.x & 31, NU = a.D / E;
    const float inv_D = 1.0f / (float)a.D;
    const bool grouped = a.group != 0;
    const int run = grouped ? a.group / E : 32, run_shift = 31 - __clz(run);
    const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
    griddep_wait();
    griddep_launch_dependents();
    uint4 vx[V], vr[RES ? V : 1];
    float2 w[V][P];
    auto fetch = [&](int64_t row) {  // units past the row are zeros
        const uint4 *px = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + row * a.ld_x);
        const uint4 *pr = RES ? reinterpret_cast<const uint4 *>(static_cast<const T *>(a.res) + row * a.ld_res) : nullptr;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = lane + 32 * j;
            vx[j] = make_uint4(0, 0, 0, 0);
            if constexpr (RES) vr[j] = make_uint4(0, 0, 0, 0);
            if (u < NU) {
                vx[j] = ld_stream(px + u);
                if constexpr (RES) vr[j] = ld_stream(pr + u);
            }
        }
    };
    int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (row < a.rows) fetch(row);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint4 c = lane + 32 * j < NU ? __ldg(static_cast<const uint4 *>(a.w) + lane + 32 * j) : make_uint4(0, 0, 0, 0);
        unpack_vec<T>(c, w[j]);
#pragma unroll
        for (int m = 0; m < P; ++m) w[j][m] = f2add(w[j][m], make_float2(a.weight_bias, a.weight_bias));
    }
    for (; row < a.rows; row += step) {
        float2 v[V][P], s2 = make_float2(0.f, 0.f);
        float part[V], top = 0.f;
        uint4 *nres = RES ? reinterpret_cast<uint4 *>(static_cast<T *>(a.nres) + row * a.ld_nres) : nullptr;
        uint8_t *out = static_cast<uint8_t *>(a.out) + row * a.ld_out;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            unpack_vec<T>(vx[j], v[j]);
            if constexpr (RES) {
                float2 r[P];
                unpack_vec<T>(vr[j], r);
#pragma unroll
                for (int m = 0; m < P; ++m) v[j][m] = f2add(v[j][m], r[m]);
            }
        }
        if (row + step < a.rows) fetch(row + step);  // (another row: nothing this one writes)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if constexpr (RES)
                if (lane + 32 * j < NU) nres[lane + 32 * j] = pack_vec<T>(v[j]);
            part[j] = 0.f;
#pragma unroll
            for (int m = 0; m < P; ++m) {
                s2 = f2fma(v[j][m], v[j][m], s2);
                v[j][m] = f2mul(v[j][m], w[j][m]);
                part[j] = max_abs(part[j], v[j][m].x, v[j][m].y);
            }
            top = max_abs(top, part[j]);
        }
        const float r = rsqrtf(group_sum<32>(s2.x + s2.y) * inv_D + a.eps);
        if (grouped) {
            run_maxima(part, run);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int u = lane + 32 * j;
                const float2 sc = q8_scale(part[j], r);
                store_codes(out + u * E, v[j], sc.y, a.whole_codes, u < NU);
                if (u < NU && (u & (run - 1)) == 0) a.scale[row * a.groups + (u >> run_shift)] = sc.x;
            }
        } else {
            const float2 sc = q8_scale(warp_max(top), r);
#pragma unroll
            for (int j = 0; j < V; ++j) store_codes(out + (lane + 32 * j) * E, v[j], sc.y, a.whole_codes, lane + 32 * j < NU);
            if (lane == 0) a.scale[row] = sc.x;
        }
    }
}

// Any row length, stride and alignment: one element a thread, the row read twice (the
// second time from L2).  Groups go to a warp each.
template <typename T, bool RES>
__global__ void __launch_bounds__(Q8_GENERIC_NT) q8_generic_kernel(const Q8Args a) {
    constexpr int NW = Q8_GENERIC_NT / 32;
    __shared__ float s_sum[NW];
    __shared__ float s_top[NW];
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
        float top = 0.f;
        for (int j0 = threadIdx.x; j0 < a.D; j0 += 64 * Q8_GENERIC_NT) {
            float part = 0.f;
            for (int i = 0, j = j0; i < 64 && j < a.D; ++i, j += Q8_GENERIC_NT) {
                const float h = h_of(j);
                part = fmaf(h, h, part);
                if (!a.group) top = max_abs(top, h * weight(j));
            }
            ss += part;
        }
        ss = group_sum<32>(ss);
        top = warp_max(top);
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
            top = warp_max(lane < NW ? s_top[lane] : 0.f);
            const float2 s = q8_scale(top, r);
            for (int j = threadIdx.x; j < a.D; j += Q8_GENERIC_NT) write(j, h_of(j), s.y);
            if (threadIdx.x == 0) a.scale[row] = s.x;
        } else {
            for (int g = warp; g < a.groups; g += NW) {
                float h[4];
                float t = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = g * a.group + 32 * i + lane;
                    const bool in = 32 * i < a.group && j < a.D;
                    h[i] = in ? h_of(j) : 0.f;
                    if (in) t = max_abs(t, h[i] * weight(j));
                }
                const float2 s = q8_scale(warp_max(t), r);
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

// Rows too long for registers, on 16-byte boundaries: read twice, the second time from
// L2, in 16-byte units (2000 x 20000 bf16 70 us, 59 %; an element at a time 188).
template <typename T, bool RES>
__global__ void __launch_bounds__(Q8_GENERIC_NT, 2) q8_long_kernel(const __grid_constant__ Q8Args a) {
    constexpr int E = vec_elems<T>(), P = vec_pairs<T>(), NT = Q8_GENERIC_NT, NW = NT / 32, V = 4;
    __shared__ float2 s_row[2][NW];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, NU = a.D / E;
    const bool grouped = a.group != 0;
    const int run = grouped ? a.group / E : 32, run_shift = 31 - __clz(run);
    const uint4 *w = static_cast<const uint4 *>(a.w);
    griddep_wait();
    griddep_launch_dependents();
    int side = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + row * a.ld_x);
        const uint4 *res = RES ? reinterpret_cast<const uint4 *>(static_cast<const T *>(a.res) + row * a.ld_res) : nullptr;
        uint4 *nres = RES ? reinterpret_cast<uint4 *>(static_cast<T *>(a.nres) + row * a.ld_nres) : nullptr;
        uint8_t *out = static_cast<uint8_t *>(a.out) + row * a.ld_out;
        // h and h w' of unit u, zeros past the row
        auto load = [&](int u, float2 (&h)[P], float2 (&v)[P]) {
            uint4 cx = make_uint4(0, 0, 0, 0), cr = cx, cw = cx;
            if (u < NU) {
                cx = x[u];
                if constexpr (RES) cr = res[u];
                cw = __ldg(w + u);
            }
            float2 r[P];
            unpack_vec<T>(cx, h);
            unpack_vec<T>(cw, v);
            if constexpr (RES) unpack_vec<T>(cr, r);
#pragma unroll
            for (int m = 0; m < P; ++m) {
                if constexpr (RES) h[m] = f2add(h[m], r[m]);
                v[m] = f2mul(h[m], f2add(v[m], make_float2(a.weight_bias, a.weight_bias)));
            }
        };
        // A sum of sums of 32 rounds, so that rounding grows with neither length alone.
        float ss = 0.f, top = 0.f;
        for (int u1 = t; u1 < NU; u1 += 32 * V * NT) {
            float some = 0.f;
            for (int u0 = u1; u0 < min(NU, u1 + 32 * V * NT); u0 += V * NT) {
                float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float2 h[P], v[P];
                    load(u0 + j * NT, h, v);
#pragma unroll
                    for (int m = 0; m < P; ++m) {
                        s2 = f2fma(h[m], h[m], s2);
                        top = max_abs(top, v[m].x, v[m].y);
                    }
                }
                some += s2.x + s2.y;
            }
            ss += some;
        }
        ss = group_sum<32>(ss);
        top = warp_max(top);
        if (lane == 0) s_row[side][warp] = make_float2(ss, top);
        __syncthreads();
        const float2 mine = s_row[side][lane & (NW - 1)];
        side ^= 1;
        const float r = rsqrtf(group_sum<NW>(mine.x) * (1.0f / (float)a.D) + a.eps);
        const float2 whole = q8_scale(run_max(mine.y, NW), r);
        if (!grouped && t == 0) a.scale[row] = whole.x;
        for (int u0 = t - lane; u0 < NU; u0 += V * NT) {  // the same in a warp's lanes
            float2 v[V][P];
            float part[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int u = u0 + lane + j * NT;
                float2 h[P];
                load(u, h, v[j]);
                if constexpr (RES)
                    if (u < NU) nres[u] = pack_vec<T>(h);
                part[j] = 0.f;
#pragma unroll
                for (int m = 0; m < P; ++m) part[j] = max_abs(part[j], v[j][m].x, v[j][m].y);
            }
            if (grouped) run_maxima(part, run);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int u = u0 + lane + j * NT;
                const float2 sc = grouped ? q8_scale(part[j], r) : whole;
                store_codes(out + (int64_t)u * E, v[j], sc.y, a.whole_codes, u < NU);
                if (grouped && u < NU && (u & (run - 1)) == 0) a.scale[row * a.groups + (u >> run_shift)] = sc.x;
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
    if (p.threads <= 128) return launch_q8_row<T, RES, SHIFT, true, Q8_UNITS, 128, 4>(p, a, s);
    if (p.threads <= 256) return launch_q8_row<T, RES, SHIFT, true, Q8_UNITS, 256, 2>(p, a, s);
    return launch_q8_row<T, RES, SHIFT, true, Q8_UNITS, 512, 1>(p, a, s);
}

template <typename T, bool RES> cudaError_t launch_q8_kind(const Q8Plan &p, const Q8Args &a, cudaStream_t s) {
    if (p.kind == Q8_GENERIC) return launch_pdl(q8_generic_kernel<T, RES>, dim3(p.grid), dim3(p.threads), 0, s, a);
    if (p.kind == Q8_LONG) return launch_pdl(q8_long_kernel<T, RES>, dim3(p.grid), dim3(p.threads), 0, s, a);
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
