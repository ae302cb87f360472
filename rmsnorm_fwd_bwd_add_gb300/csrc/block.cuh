// block.cuh -- the norm pair around a block for rows that fit on chip.
//
// HBM-bound: the forward moves four row tensors, the VJP up to six, each once.
// A row's elements sit in registers, UNITS units a thread, from the one read to
// the outputs; both norms' sums cross the CTA through one barrier each.
//
//   BLOCK_STAGED  one row a CTA at a time out of a shared-memory ring that thread
//                 0 fills with 1-D bulk copies `stages` rows ahead, so that the
//                 barriers of a row hide behind the copies of the next ones.  A
//                 row off 16-byte boundaries is copied as its aligned superset.
//                 A stage is free again once every thread has its units in
//                 registers, at the row's first barrier.
//   BLOCK_DIRECT  one row a CTA, loaded from global memory: no more rows than
//                 CTAs fit at once, where a ring has nothing to run ahead of.
//   BLOCK_WARP    one row a warp (short rows): no barriers; several rows a CTA.
//
// Per-thread state: w1 = weight_bias + w_pre and m = scale * gate * (weight_bias
// + w_post) of its columns in fp32 (m is rebuilt when the CTA's rows pass to
// another gate row; with a gate row per row, the gate streams with the row and
// m holds the rest), the VJP's two accumulators of its columns.
#pragma once

#include "block.h"
#include "units.cuh"

namespace rmsn {

// Elements a thread owns: 32 bytes of a row in 16-byte or 4-byte units of 16-bit
// types; 8 elements otherwise.
template <typename T, int UB> __host__ __device__ constexpr int block_units() {
    return sizeof(T) == 2 && UB >= 4 ? 16 / unit_elems<T, UB>() : 8 / unit_elems<T, UB>();
}
template <typename T, int UB> __host__ __device__ constexpr int block_elems() {
    return block_units<T, UB>() * unit_elems<T, UB>();
}

constexpr int BLOCK_MAX_STAGES = 8;
constexpr int BLOCK_HEADER = 128;  // the ring's mbarriers, ahead of its data

// Sums of N values over the CTA's `nw` warps (at most MAXW), the same in every
// thread; `red` holds N floats a warp.  Returns false if any thread passed !ok.
template <int N, int MAXW>
__device__ __forceinline__ bool cta_sums(float (&v)[N], float (*red)[4], int nw, bool ok) {
    constexpr int WP = MAXW <= 4 ? 4 : MAXW <= 8 ? 8 : MAXW <= 16 ? 16 : 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = group_sum<32>(v[i]);
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) red[warp][i] = v[i];
    }
    const bool bad = __syncthreads_or(!ok);
    const int w = lane & (WP - 1);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = group_sum<WP>(w < nw ? red[w][i] : 0.f);
    return !bad;
}

// The ring of one CTA: rows r0, r0 + 1, ... of N tensors.
struct BlockRing {
    uint64_t *full;
    unsigned char *data;
    int S;
    uint32_t stage_bytes;  // of one tensor
    int tensors;
};

template <typename T>
__device__ __forceinline__ void ring_issue(const BlockRing &ring, const BlockArgs &a, const void *const (&src)[5],
                                           const int64_t (&ld)[5], int64_t row, int stage, uint64_t policy) {
    if (row == a.drop_row) return;
    const uint32_t bytes = (uint32_t)a.D * (uint32_t)sizeof(T);
    uint32_t total = 0;
#pragma unroll
    for (int t = 0; t < 5; ++t)
        if (src[t]) {
            const uintptr_t p = (uintptr_t)(static_cast<const T *>(src[t]) + row * ld[t]);
            total += ((uint32_t)(p & 15u) + bytes + 15u) & ~15u;
        }
    mbar_arrive_expect_tx(&ring.full[stage], total);
    unsigned char *dst = ring.data + (size_t)stage * ring.tensors * ring.stage_bytes;
#pragma unroll
    for (int t = 0; t < 5; ++t)
        if (src[t]) {
            const uintptr_t p = (uintptr_t)(static_cast<const T *>(src[t]) + row * ld[t]);
            const uint32_t off = (uint32_t)(p & 15u);
            bulk_g2s(dst, reinterpret_cast<const void *>(p - off), (off + bytes + 15u) & ~15u, &ring.full[stage],
                     policy);
            dst += ring.stage_bytes;
        }
}

// Forward -----------------------------------------------------------------
template <typename T, int UB, int MAXT, int MINB, int KIND, bool GROW>
__global__ void __launch_bounds__(MAXT, MINB) block_fwd_kernel(const __grid_constant__ BlockArgs a) {
    using Raw = typename RawUnit<UB>::type;
    constexpr int E = unit_elems<T, UB>(), V = block_units<T, UB>(), MAXW = MAXT / 32;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float s_red[2][KIND == BLOCK_WARP ? 1 : MAXW][4];
    const int NT = KIND == BLOCK_WARP ? 32 : (int)blockDim.x;
    const int t0 = KIND == BLOCK_WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    const int R = KIND == BLOCK_WARP ? (int)(blockDim.x >> 5) : 1;
    const int NU = a.D / E, nw = (int)(blockDim.x >> 5);
    const float inv_D = 1.0f / (float)a.D;
    constexpr bool per_row = GROW;  // a gate row for each row
    const bool post = a.w_post != nullptr;
    const int64_t r0 = first_row(blockIdx.x, gridDim.x, a.rows), r1 = first_row(blockIdx.x + 1, gridDim.x, a.rows);

    const void *src[5] = {a.y, a.res, per_row ? a.gate : nullptr, nullptr, nullptr};
    const int64_t ld[5] = {a.ld_y, a.ld_res, a.ld_gate, 0, 0};
    BlockRing ring{reinterpret_cast<uint64_t *>(smem), smem + BLOCK_HEADER, a.stages, a.stage_bytes, per_row ? 3 : 2};
    uint64_t policy = 0;
    if constexpr (KIND == BLOCK_STAGED) {
        policy = l2_evict_first_policy();
        if (threadIdx.x == 0) {
            for (int s = 0; s < ring.S; ++s) mbar_init(&ring.full[s], 1);
            fence_mbar_init();
        }
        __syncthreads();
    }
    griddep_wait();
    if constexpr (KIND == BLOCK_STAGED) {
        if (threadIdx.x == 0)
            for (int s = 0; s < ring.S && r0 + s < r1; ++s) ring_issue<T>(ring, a, src, ld, r0 + s, s, policy);
    }

    // w1, and m without the gate
    float w1[V][E], m[V][E];
    auto load_unit = [&](const void *base, int u, float (&f)[E]) {
        unpack_unit<T, UB>(static_cast<const Raw *>(base)[u], f);
    };
    auto load_m = [&](const T *gate_row) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = t0 + j * NT;
            if (u < NU) {
                float f[E], q[E];
                if (post) load_unit(a.w_post, u, f);
                if (gate_row) load_unit(gate_row, u, q);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    m[j][e] = (post ? a.weight_bias + f[e] : 1.f) * (gate_row ? a.scale * q[e] : a.scale);
            }
        }
    };
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int u = t0 + j * NT;
        if (u < NU) {
            float f[E];
            load_unit(a.w_pre, u, f);
#pragma unroll
            for (int e = 0; e < E; ++e) w1[j][e] = a.weight_bias + f[e];
        }
    }
    if (!a.gate || per_row) load_m(nullptr);

    int64_t group_end = a.gate && !per_row ? r0 : INT64_MAX;  // first row past the gate row held in m
    int s = 0;
    uint32_t ph = 0;
    for (int64_t row = r0 + (KIND == BLOCK_WARP ? (int)(threadIdx.x >> 5) : 0); row < r1; row += R) {
        if (row >= group_end) {
            const int64_t gr = row / a.rows_per_gate;
            group_end = (gr + 1) * a.rows_per_gate;
            load_m(static_cast<const T *>(a.gate) + gr * a.ld_gate);
        }
        const T *py = static_cast<const T *>(a.y) + row * a.ld_y;
        const T *pr = static_cast<const T *>(a.res) + row * a.ld_res;
        const T *pg = per_row ? static_cast<const T *>(a.gate) + row * a.ld_gate : nullptr;
        bool ok = true;
        if constexpr (KIND == BLOCK_STAGED) {  // the same rows in the stage
            const unsigned char *st = ring.data + (size_t)s * ring.tensors * ring.stage_bytes;
            py = reinterpret_cast<const T *>(st + ((uintptr_t)py & 15u));
            pr = reinterpret_cast<const T *>(st + ring.stage_bytes + ((uintptr_t)pr & 15u));
            if (per_row) pg = reinterpret_cast<const T *>(st + 2 * ring.stage_bytes + ((uintptr_t)pg & 15u));
            ok = mbar_wait_bounded(&ring.full[s], ph, a.wait_budget);
        }
        Raw vy[V], vr[V];
        float v[V][E];  // m * y, the added term before r_y
        float sum[1] = {0.f};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = t0 + j * NT;
            if (u < NU) {
                vy[j] = reinterpret_cast<const Raw *>(py)[u];
                vr[j] = reinterpret_cast<const Raw *>(pr)[u];
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = t0 + j * NT;
            if (u < NU) {
                float f[E];
                unpack_unit<T, UB>(vy[j], f);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    sum[0] = fmaf(f[e], f[e], sum[0]);
                    v[j][e] = m[j][e] * f[e];
                }
                if constexpr (GROW) {
                    float q[E];
                    load_unit(pg, u, q);
#pragma unroll
                    for (int e = 0; e < E; ++e) v[j][e] *= q[e];
                }
            }
        }
        if constexpr (KIND == BLOCK_WARP) {
            sum[0] = group_sum<32>(sum[0]);
        } else {
            ok = cta_sums<1, MAXW>(sum, s_red[0], nw, ok);
        }
        if constexpr (KIND == BLOCK_STAGED) {
            if (!ok) {  // leave once this CTA's copies have landed
                if (threadIdx.x == 0) {
                    atomicOr(a.status, DEVSTATUS_WAIT_TIMEOUT);
                    for (int64_t k = row; k < r1 && k < row + ring.S; ++k) {
                        const int64_t i = k - r0;
                        if (k != a.drop_row)
                            mbar_wait_bounded(&ring.full[i % ring.S], (uint32_t)((i / ring.S) & 1), DEFAULT_WAIT_BUDGET);
                    }
                }
                return;
            }
            // every thread has its units of this stage in registers
            if (threadIdx.x == 0 && row + ring.S < r1) ring_issue<T>(ring, a, src, ld, row + ring.S, s, policy);
        }
        const float r_y = post ? rsqrtf(sum[0] * inv_D + a.eps) : 1.f;
        sum[0] = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = t0 + j * NT;
            if (u < NU) {
                float f[E];
                unpack_unit<T, UB>(vr[j], f);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    v[j][e] = fmaf(v[j][e], r_y, f[e]);  // h
                    sum[0] = fmaf(v[j][e], v[j][e], sum[0]);
                }
            }
        }
        if constexpr (KIND == BLOCK_WARP) {
            sum[0] = group_sum<32>(sum[0]);
        } else {
            cta_sums<1, MAXW>(sum, s_red[1], nw, true);
        }
        const float r_h = rsqrtf(sum[0] * inv_D + a.eps);
        Raw *out = reinterpret_cast<Raw *>(static_cast<T *>(a.out0) + row * a.ld_out0);
        Raw *nres = reinterpret_cast<Raw *>(static_cast<T *>(a.out1) + row * a.ld_out1);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = t0 + j * NT;
            if (u < NU) {
                nres[u] = pack_unit<T, UB>(v[j]);
                float o[E];
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = v[j][e] * r_h * w1[j][e];
                out[u] = pack_unit<T, UB>(o);
            }
        }
        if (a.rstd && t0 == 0) {
            a.rstd[row] = r_y;
            a.rstd[a.rows + row] = r_h;
        }
        if constexpr (KIND == BLOCK_STAGED) {
            if (++s == ring.S) {
                s = 0;
                ph ^= 1u;
            }
        }
    }
    griddep_launch_dependents();
}

// VJP -----------------------------------------------------------------------
// Hides from the compiler that a register's value is unchanged, so that units
// kept across a barrier stay packed and are unpacked again behind it (bf16: 8
// registers a tensor instead of 16; without it the VJP spills 208 bytes).
__device__ __forceinline__ void keep_packed(uint4 &v) {
    asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w));
}
__device__ __forceinline__ void keep_packed(uint32_t &) {}
__device__ __forceinline__ void keep_packed(uint16_t &) {}

// E consecutive floats; a unit's floats start on a 16-byte boundary when E >= 4.
template <int E>
__device__ __forceinline__ void store_floats(float *p, const float (&f)[E]) {
    if constexpr (E >= 4) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i)
            reinterpret_cast<float4 *>(p)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) p[e] = f[e];
    }
}

template <typename T, int UB, int MAXT, int MINB, int KIND, bool GROW>
__global__ void __launch_bounds__(MAXT, MINB) block_vjp_kernel(const __grid_constant__ BlockArgs a) {
    using Raw = typename RawUnit<UB>::type;
    constexpr int E = unit_elems<T, UB>(), V = block_units<T, UB>(), MAXW = MAXT / 32;
    // 16-byte units stay in registers; smaller ones take a register each and are
    // read from the stage (or L1) again instead.
    constexpr bool HOLD = UB == 16;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float s_red[2][KIND == BLOCK_WARP ? 1 : MAXW][4];
    const int NT = KIND == BLOCK_WARP ? 32 : (int)blockDim.x;
    const int t0 = KIND == BLOCK_WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    const int R = KIND == BLOCK_WARP ? (int)(blockDim.x >> 5) : 1;
    const int ry = KIND == BLOCK_WARP ? (int)(threadIdx.x >> 5) : 0;
    const int D = a.D, NU = D / E, nw = (int)(blockDim.x >> 5);
    const float inv_D = 1.0f / (float)D;
    constexpr bool per_row = GROW;  // a gate row for each row
    const bool post = a.w_post != nullptr, more = a.g_res != nullptr;
    const bool saved = a.rstd != nullptr;
    const int64_t cta = blockIdx.x, grid = gridDim.x;
    const int64_t r0 = first_row(cta, grid, a.rows), r1 = first_row(cta + 1, grid, a.rows);

    const void *src[5] = {a.y, a.res, a.g, a.g_res, per_row ? a.gate : nullptr};
    const int64_t ld[5] = {a.ld_y, a.ld_res, a.ld_g, a.ld_g_res, a.ld_gate};
    BlockRing ring{reinterpret_cast<uint64_t *>(smem), smem + BLOCK_HEADER, a.stages, a.stage_bytes, 3 + more + per_row};
    uint64_t policy = 0;
    if constexpr (KIND == BLOCK_STAGED) {
        policy = l2_evict_first_policy();
        if (threadIdx.x == 0) {
            for (int s = 0; s < ring.S; ++s) mbar_init(&ring.full[s], 1);
            fence_mbar_init();
        }
        __syncthreads();
    }
    griddep_wait();
    if constexpr (KIND == BLOCK_STAGED) {
        if (threadIdx.x == 0)
            for (int s = 0; s < ring.S && r0 + s < r1; ++s) ring_issue<T>(ring, a, src, ld, r0 + s, s, policy);
    }

    float w1[V][E], m[V][E], acc_pre[V][E], acc_mid[V][E];
    auto load_unit = [&](const void *base, int u, float (&f)[E]) {
        unpack_unit<T, UB>(static_cast<const Raw *>(base)[u], f);
    };
    auto load_m = [&](const T *gate_row) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = t0 + j * NT;
            if (u < NU) {
                float f[E], q[E];
                if (post) load_unit(a.w_post, u, f);
                if (gate_row) load_unit(gate_row, u, q);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    m[j][e] = (post ? a.weight_bias + f[e] : 1.f) * (gate_row ? a.scale * q[e] : a.scale);
            }
        }
    };
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int u = t0 + j * NT;
        float f[E];
        if (u < NU) load_unit(a.w_pre, u, f);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            w1[j][e] = u < NU ? a.weight_bias + f[e] : 0.f;
            acc_pre[j][e] = acc_mid[j][e] = 0.f;
        }
    }
    if (!a.gate || per_row) load_m(nullptr);

    // Adds the warps' accumulators (BLOCK_WARP) in warp order and writes the row.
    auto flush = [&](float (&acc)[V][E], float *dst) {
        if constexpr (KIND == BLOCK_WARP) {
            float *buf = reinterpret_cast<float *>(smem);  // [R][D]
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int u = t0 + j * NT;
                if (u < NU) store_floats<E>(buf + (size_t)ry * D + u * E, acc[j]);
            }
            __syncthreads();
            for (int c = threadIdx.x; c < D; c += blockDim.x) {
                float t = buf[c];
                for (int k = 1; k < R; ++k) t += buf[(size_t)k * D + c];
                dst[c] = t;
            }
            __syncthreads();  // buf may be written again
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int u = t0 + j * NT;
                if (u < NU) store_floats<E>(dst + (size_t)u * E, acc[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[j][e] = 0.f;
    };

    int s = 0;
    uint32_t ph = 0;
    for (int64_t seg = r0; seg < r1;) {  // rows of one gate row
        const int64_t gr = per_row ? 0 : seg / a.rows_per_gate;
        const int64_t g_end = per_row ? a.rows : (gr + 1) * a.rows_per_gate;
        const int64_t end = min(r1, g_end);
        if (a.gate && !per_row) load_m(static_cast<const T *>(a.gate) + gr * a.ld_gate);
        for (int64_t row = seg + ry; row < end; row += R) {
            float r_y = 1.f, r_h = 0.f;
            if (saved) {
                if (post) r_y = __ldg(a.rstd + row);
                r_h = __ldg(a.rstd + a.rows + row);
            }
            const T *py = static_cast<const T *>(a.y) + row * a.ld_y;
            const T *phh = static_cast<const T *>(a.res) + row * a.ld_res;
            const T *pgo = static_cast<const T *>(a.g) + row * a.ld_g;
            const T *pgr = more ? static_cast<const T *>(a.g_res) + row * a.ld_g_res : nullptr;
            const T *pga = per_row ? static_cast<const T *>(a.gate) + row * a.ld_gate : nullptr;
            bool ok = true;
            if constexpr (KIND == BLOCK_STAGED) {
                const unsigned char *st = ring.data + (size_t)s * ring.tensors * ring.stage_bytes;
                auto staged = [&](const T *p) {
                    const T *q = reinterpret_cast<const T *>(st + ((uintptr_t)p & 15u));
                    st += ring.stage_bytes;
                    return q;
                };
                py = staged(py);
                phh = staged(phh);
                pgo = staged(pgo);
                if (more) pgr = staged(pgr);
                if (per_row) pga = staged(pga);
                ok = mbar_wait_bounded(&ring.full[s], ph, a.wait_budget);
            }
            Raw vy[V], vh[V], vg[V], vr[V], va[GROW ? V : 1];
            auto fetch = [&](const T *p, Raw *v) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int u = t0 + j * NT;
                    if (u < NU) v[j] = reinterpret_cast<const Raw *>(p)[u];
                }
            };
            if constexpr (HOLD) {
                fetch(py, vy);
                fetch(phh, vh);
                fetch(pgo, vg);
                if (more) fetch(pgr, vr);
                if constexpr (GROW) fetch(pga, va);
            }
            auto repack = [&]() {
                if constexpr (HOLD && sizeof(T) == 2) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        keep_packed(vy[j]);
                        keep_packed(vh[j]);
                        keep_packed(vg[j]);
                    }
                }
            };
            // unit j of a row, from the registers or from where it was staged
            auto get = [&](const T *p, const Raw *v, int j, float (&f)[E]) {
                if constexpr (HOLD) unpack_unit<T, UB>(v[j], f);
                else unpack_unit<T, UB>(reinterpret_cast<const Raw *>(p)[t0 + j * NT], f);
            };
            float sum[3] = {0.f, 0.f, 0.f};  // g w1 h, h^2, y^2
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (t0 + j * NT < NU) {
                    float fh[E], fg[E];
                    get(phh, vh, j, fh);
                    get(pgo, vg, j, fg);
#pragma unroll
                    for (int e = 0; e < E; ++e) sum[0] = fmaf(fg[e] * w1[j][e], fh[e], sum[0]);
                    if (!saved) {
                        float fy[E];
                        get(py, vy, j, fy);
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            sum[1] = fmaf(fh[e], fh[e], sum[1]);
                            sum[2] = fmaf(fy[e], fy[e], sum[2]);
                        }
                    }
                }
            }
            if constexpr (KIND == BLOCK_WARP) {
#pragma unroll
                for (int i = 0; i < 3; ++i) sum[i] = group_sum<32>(sum[i]);
            } else {
                ok = cta_sums<3, MAXW>(sum, s_red[0], nw, ok);
            }
            if constexpr (KIND == BLOCK_STAGED) {
                if (!ok) {
                    if (threadIdx.x == 0) {
                        atomicOr(a.status, DEVSTATUS_WAIT_TIMEOUT);
                        for (int64_t k = row; k < r1 && k < row + ring.S; ++k) {
                            const int64_t i = k - r0;
                            if (k != a.drop_row)
                                mbar_wait_bounded(&ring.full[i % ring.S], (uint32_t)((i / ring.S) & 1),
                                                  DEFAULT_WAIT_BUDGET);
                        }
                    }
                    return;
                }
                if (HOLD && threadIdx.x == 0 && row + ring.S < r1)
                    ring_issue<T>(ring, a, src, ld, row + ring.S, s, policy);
            }
            repack();
            if (!saved) {
                r_h = rsqrtf(sum[1] * inv_D + a.eps);
                if (post) r_y = rsqrtf(sum[2] * inv_D + a.eps);
            }
            const float cc = (r_h * r_h) * (sum[0] * inv_D);
            // g_h of unit j
            auto grad_h = [&](int j, const float (&fh)[E], const float (&fg)[E], float (&o)[E]) {
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = r_h * (fg[e] * w1[j][e] - fh[e] * cc);
                if (more) {
                    float fr[E];
                    get(pgr, vr, j, fr);
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] += fr[e];
                }
            };
            auto mult = [&](int j, float (&mm)[E]) {
#pragma unroll
                for (int e = 0; e < E; ++e) mm[e] = m[j][e];
                if constexpr (GROW) {
                    float q[E];
                    get(pga, va, j, q);
#pragma unroll
                    for (int e = 0; e < E; ++e) mm[e] *= q[e];
                }
            };
            sum[0] = 0.f;
            if (post) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (t0 + j * NT < NU) {
                        float fh[E], fg[E], fy[E], o[E], mm[E];
                        get(phh, vh, j, fh);
                        get(pgo, vg, j, fg);
                        get(py, vy, j, fy);
                        grad_h(j, fh, fg, o);
                        mult(j, mm);
#pragma unroll
                        for (int e = 0; e < E; ++e) sum[0] = fmaf(mm[e] * o[e], fy[e], sum[0]);
                    }
                }
                float one[1] = {sum[0]};
                if constexpr (KIND == BLOCK_WARP) one[0] = group_sum<32>(one[0]);
                else cta_sums<1, MAXW>(one, s_red[1], nw, true);
                sum[0] = one[0];
            }
            repack();
            const float ee = (r_y * r_y) * (sum[0] * inv_D);
            Raw *gy = reinterpret_cast<Raw *>(static_cast<T *>(a.out0) + row * a.ld_out0);
            Raw *gh = reinterpret_cast<Raw *>(static_cast<T *>(a.out1) + row * a.ld_out1);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int u = t0 + j * NT;
                if (u < NU) {
                    float fh[E], fg[E], fy[E], o[E], mm[E], q[E];
                    get(phh, vh, j, fh);
                    get(pgo, vg, j, fg);
                    get(py, vy, j, fy);
                    grad_h(j, fh, fg, o);
                    mult(j, mm);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        acc_pre[j][e] = fmaf(fg[e], fh[e] * r_h, acc_pre[j][e]);
                        q[e] = o[e] * (fy[e] * r_y);  // g_h y r_y
                    }
                    if constexpr (GROW) {  // this row is its gate row: finished here, and gw_post's term weighted
                        float ga[E], w2[E];
                        get(pga, va, j, ga);
                        if (post) load_unit(a.w_post, u, w2);
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            acc_mid[j][e] = fmaf(q[e], a.scale * ga[e], acc_mid[j][e]);
                            w2[e] = q[e] * a.scale * (post ? a.weight_bias + w2[e] : 1.f);
                        }
                        store_floats<E>(a.g_gate + row * D + (size_t)u * E, w2);
                    } else {
#pragma unroll
                        for (int e = 0; e < E; ++e) acc_mid[j][e] = fmaf(q[e], a.scale, acc_mid[j][e]);
                    }
                    gh[u] = pack_unit<T, UB>(o);
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] = r_y * (mm[e] * o[e] - fy[e] * ee);
                    gy[u] = pack_unit<T, UB>(o);
                }
            }
            if constexpr (KIND == BLOCK_STAGED) {
                if constexpr (!HOLD) {  // the stage is read until here
                    __syncthreads();
                    if (threadIdx.x == 0 && row + ring.S < r1)
                        ring_issue<T>(ring, a, src, ld, row + ring.S, s, policy);
                }
                if (++s == ring.S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (a.gate || post) {
            const bool whole = a.g_gate && !per_row && gr * a.rows_per_gate >= r0 && g_end <= r1;
            flush(acc_mid, per_row ? a.part_mid + 2 * cta * D
                           : whole ? a.g_gate + gr * D
                                   : a.part_mid + mid_slot(cta, gr, grid, a.rows, a.rows_per_gate) * D);
        }
        seg = end;
    }
    flush(acc_pre, a.part_pre + cta * D);
    griddep_launch_dependents();
}

}  // namespace rmsn
