// block.cuh -- the norm pair around a block for rows that fit on chip.
//
// HBM-bound: the forward moves four row tensors, the VJP up to six, each once.
// A row's elements sit in registers, 32 bytes of each tensor a thread, from the
// one read to the outputs, and all of a row's sums cross the CTA through one
// barrier, although the second norm's depends on the first's:
//   forward: with v = m y, m = scale * gate * w2, sum h^2 = sum res^2 + 2 r_y sum
//     res v + r_y^2 sum v^2.  Where the block nearly undoes the stream (the
//     result is below an eighth of its terms), or v^2 is out of fp32's range, it is
//     summed again from h itself.
//   VJP: sum m g_h y = r_h (sum u g w1 - c sum u h) + sum u g_res, u = m y: the
//     same terms as its own sum has, so no digits are lost.  u g w1 and u h must
//     stay in fp32's range (a second way through, as in the forward, cost the
//     instances without a FORM 150 to 500 bytes of spills a thread).
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
// w1 = weight_bias + w_pre sits in shared memory in fp32 (in registers the VJP
// spilled), or packed in registers where a thread sees few rows.  In registers,
// for a thread's columns: m = scale * gate * (weight_bias + w_post), rebuilt when
// the CTA's rows pass to another gate row (with a gate row per row, the gate
// streams with the row and m holds the rest), and the VJP's two accumulators.
//
// A row's units are 16 bytes where its address and length allow.  Where they do
// not but all row tensors stand alike to 16-byte boundaries (dense rows of an odd
// D), SHIFT takes the 16-byte units of memory: a CTA's rows all stand the same way,
// so its columns are fixed as ever, and the columns before a row's first boundary and
// behind its last unit are an element a thread of the first warp or two.  (Masking
// the cut units instead made their warps late for every barrier: 40.3 us against 28.7
// for 5000 x 4097.)  Only tensors that stand differently, and rows of a warp, are
// read in units of 4 or 2 bytes.
//
// On the GB300 (6.7 TB/s copied), inputs changing from call to call: forward of 16384 x
// 8192 bf16 with 8 gate rows 166 us (96 % of that), 5000 x 4097 fp16 31.5 us (78 %); VJP of
// 16384 x 4096 bf16 135 us (89 %: 123 registers a thread leave an SM 16 warps, and the last
// 5 us are the second stage), 4095 x 2048 fp32 with a gate row each 42.6 us (82 %), 16384 x
// 512 31 us (48 %: no ring, and 16 warps an SM do not hide a row's trip to memory), 8192 x
// 16384 517 us (46 %: rows of 513 threads or more leave the ring one or two stages and a
// thread 64 registers, which spill).
#pragma once

#include <cfloat>
#include <type_traits>

#include "block.h"
#include "units.cuh"

namespace rmsn {

// A thread owns 32 bytes of a row as SLOTS slots of P float2 pairs, the operands of
// packed fp32x2 arithmetic.  A slot is one unit, or, for one-element units, two
// of them a CTA's width apart (its second may lie past the row: it reads 0 and
// is not written).  `raw` keeps a slot's elements packed.
template <typename T, int UB> struct Slot {
    static constexpr int E = unit_elems<T, UB>();
    static constexpr int P = E > 1 ? E / 2 : 1;
    static constexpr int COUNT = 32 / (int)sizeof(T) / (2 * P);
    using Unit = typename RawUnit<UB>::type;
    struct Two { uint32_t a, b; };  // two fp32 units
    using Raw = typename std::conditional<(E > 1), Unit,
                                          typename std::conditional<sizeof(T) == 4, Two, uint32_t>::type>::type;

    // First unit of slot j of thread t among NT; whether the slot has any.
    static __device__ __forceinline__ int unit(int j, int t, int NT) { return t + (E > 1 ? j : 2 * j) * NT; }

    static __device__ __forceinline__ Raw load(const void *row, int u, int NT, int NU) {
        const Unit *p = static_cast<const Unit *>(row);
        if constexpr (E > 1) {
            return p[u];
        } else if constexpr (sizeof(T) == 4) {
            return Two{p[u], u + NT < NU ? p[u + NT] : 0u};
        } else {
            return (uint32_t)p[u] | (u + NT < NU ? (uint32_t)p[u + NT] << 16 : 0u);
        }
    }
    static __device__ __forceinline__ void unpack(const Raw &v, float2 (&f)[P]) {
        if constexpr (E > 2) {
            unpack_vec<T>(v, f);
        } else if constexpr (sizeof(T) == 4) {
            f[0] = make_float2(__uint_as_float(v.a), __uint_as_float(v.b));
        } else {
            f[0] = Cvt<T>::unpack2(v);
        }
    }
    static __device__ __forceinline__ void store(void *row, int u, int NT, int NU, const float2 (&f)[P]) {
        Unit *p = static_cast<Unit *>(row);
        if constexpr (E > 2) {
            p[u] = pack_vec<T>(f);
        } else if constexpr (E == 2) {
            p[u] = Cvt<T>::pack2(f[0].x, f[0].y);
        } else if constexpr (sizeof(T) == 4) {
            p[u] = __float_as_uint(f[0].x);
            if (u + NT < NU) p[u + NT] = __float_as_uint(f[0].y);
        } else {
            const uint32_t v = Cvt<T>::pack2(f[0].x, f[0].y);
            p[u] = (uint16_t)v;
            if (u + NT < NU) p[u + NT] = (uint16_t)(v >> 16);
        }
    }
    // The slot's elements as floats at their columns of an fp32 row (16-byte
    // aligned where a unit has four elements or more).
    static __device__ __forceinline__ void store_floats(float *row, int u, int NT, int NU, const float2 (&f)[P], float k) {
        if constexpr (E >= 4) {
#pragma unroll
            for (int i = 0; i < E / 4; ++i)
                reinterpret_cast<float4 *>(row + (size_t)u * E)[i] =
                    make_float4(f[2 * i].x * k, f[2 * i].y * k, f[2 * i + 1].x * k, f[2 * i + 1].y * k);
        } else if constexpr (E == 2) {
            row[2 * u] = f[0].x * k;
            row[2 * u + 1] = f[0].y * k;
        } else {
            row[u] = f[0].x * k;
            if (u + NT < NU) row[u + NT] = f[0].y * k;
        }
    }
    // The same for a slot whose columns start at `c`, on no boundary (16-byte units).
    static __device__ __forceinline__ Raw load_columns(const T *p, int c) {
        T t[E];
#pragma unroll
        for (int e = 0; e < E; ++e) t[e] = p[c + e];
        Raw v;
        memcpy(&v, t, sizeof(v));
        return v;
    }
    static __device__ __forceinline__ void store_floats_at(float *row, int c, const float2 (&f)[P], float k) {
#pragma unroll
        for (int e = 0; e < E; ++e) row[c + e] = (e & 1 ? f[e / 2].y : f[e / 2].x) * k;
    }
    // A per-column table in shared memory, laid out so that a warp's lanes read
    // consecutive 16- or 8-byte words: [pairs of pairs][units] (E >= 4), [units].
    static __device__ __forceinline__ void put(float *tab, int u, int NT, int NU, const float2 (&f)[P]) {
        if constexpr (E >= 4) {
#pragma unroll
            for (int i = 0; i < E / 4; ++i)
                reinterpret_cast<float4 *>(tab)[i * NU + u] = make_float4(f[2 * i].x, f[2 * i].y, f[2 * i + 1].x, f[2 * i + 1].y);
        } else if constexpr (E == 2) {
            reinterpret_cast<float2 *>(tab)[u] = f[0];
        } else {
            tab[u] = f[0].x;
            if (u + NT < NU) tab[u + NT] = f[0].y;
        }
    }
    static __device__ __forceinline__ void get(const float *tab, int u, int NT, int NU, float2 (&f)[P]) {
        if constexpr (E >= 4) {
#pragma unroll
            for (int i = 0; i < E / 4; ++i) {
                const float4 v = reinterpret_cast<const float4 *>(tab)[i * NU + u];
                f[2 * i] = make_float2(v.x, v.y);
                f[2 * i + 1] = make_float2(v.z, v.w);
            }
        } else if constexpr (E == 2) {
            f[0] = reinterpret_cast<const float2 *>(tab)[u];
        } else {
            f[0] = make_float2(tab[u], u + NT < NU ? tab[u + NT] : 0.f);
        }
    }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Shared memory of BLOCK_STAGED: the ring's mbarriers (BLOCK_HEADER), the table w1,
// the ring.

// Sums of four (N <= 4) or eight (N <= 8) values over a warp at once.  The first
// steps halve the number of values a lane carries instead of summing each over
// all lanes: 2 + 1 + 1 + 1 + 1 shuffles for four values where one butterfly each
// takes 20.  Lane l ends with the sum of value l % K over the warp, the same bits
// in every lane that has it.
template <int K>
__device__ __forceinline__ float spread_sums(float (&v)[K]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = K / 2; h > 0; h /= 2) {  // lanes with bit h keep the upper h values
        const bool up = lane & h;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float give = up ? v[i] : v[i + h], keep = up ? v[i + h] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, h);
        }
    }
    float t = v[0];
#pragma unroll
    for (int off = K; off < 32; off *= 2) t += __shfl_xor_sync(0xffffffffu, t, off);
    return t;
}

template <int N> __host__ __device__ constexpr int spread_of() { return N <= 1 ? 1 : N <= 4 ? 4 : 8; }

// Sums of N values over a warp, the same in every lane.
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N]) {
    constexpr int K = spread_of<N>();
    float x[K];
#pragma unroll
    for (int i = 0; i < K; ++i) x[i] = i < N ? v[i < N ? i : 0] : 0.f;
    const float t = spread_sums<K>(x);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, t, i);
}

// Sums of N values over the CTA's `nw` warps (at most MAXW), the same in every
// thread; `red` holds eight floats a warp.  Returns false if any thread passed
// !ok.
template <int N, int MAXW>
__device__ __forceinline__ bool cta_sums(float (&v)[N], float (*red)[8], int nw, bool ok) {
    constexpr int K = spread_of<N>(), ROWS = 32 / K;  // warps a step covers
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float x[K];
#pragma unroll
    for (int i = 0; i < K; ++i) x[i] = i < N ? v[i < N ? i : 0] : 0.f;
    const float t = spread_sums<K>(x);
    if (lane < K) red[warp][lane] = t;
    const bool bad = __syncthreads_or(!ok);
    float s = 0.f;  // value lane % K of warps lane / K, lane / K + ROWS, ...
#pragma unroll
    for (int w0 = 0; w0 < MAXW; w0 += ROWS) {
        const int w = w0 + lane / K;
        if (w < nw) s += red[w][lane % K];
    }
#pragma unroll
    for (int off = K; off < 32; off *= 2) s += __shfl_xor_sync(0xffffffffu, s, off);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, s, i);
    return !bad;
}

// A float of the cluster's CTA `rank`, at the place that `p` is in this one's
// shared memory.
__device__ __forceinline__ float load_remote(const float *p, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(dsmem_addr(p, rank)) : "memory");
    return v;
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

// Hides from the compiler that a register's value is unchanged, so that units
// kept across a barrier stay packed and are unpacked again behind it (bf16: 8
// registers a tensor instead of 16).
__device__ __forceinline__ void keep_packed(uint4 &v) {
    asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w));
}
__device__ __forceinline__ void keep_packed(uint32_t &v) { asm volatile("" : "+r"(v)); }
template <typename V> __device__ __forceinline__ void keep_packed(V &v) {
    asm volatile("" : "+r"(v.a), "+r"(v.b));
}

// Forward -----------------------------------------------------------------
template <typename T, int UB, int MAXT, int MINB, int KIND, bool GROW, bool SHIFT>
__global__ void __launch_bounds__(MAXT, MINB) block_fwd_kernel(const __grid_constant__ BlockArgs a) {
    using SL = Slot<T, UB>;
    using Raw = typename SL::Raw;
    constexpr int E = SL::E, V = SL::COUNT, P = SL::P, MAXW = MAXT / 32;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float s_red[2][KIND == BLOCK_WARP ? 1 : MAXW][8];
    const int NT = KIND == BLOCK_WARP ? 32 : (int)blockDim.x;
    const int t0 = KIND == BLOCK_WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    const int R = KIND == BLOCK_WARP ? (int)(blockDim.x >> 5) : 1;
    const int D = a.D, nw = (int)(blockDim.x >> 5);
    const float inv_D = 1.0f / (float)D;
    constexpr bool per_row = GROW;  // a gate row for each row
    const bool post = a.w_post != nullptr;
    const RowDeal deal = fwd_rows(a, blockIdx.x, gridDim.x);
    // SHIFT: `hd` columns before a row's first 16-byte boundary, the same for all of
    // this CTA's rows; thread t0 also has column cx, one of those or of the rest behind
    // the last unit.
    const int hd = SHIFT ? (int)(-((uintptr_t)(static_cast<const T *>(a.y) + deal.row(0) * a.ld_y)) & 15u) / (int)sizeof(T) : 0;
    const int NU = SHIFT ? min((D - hd) / E, V * NT) : D / E;
    const int cx = !SHIFT || t0 >= D - NU * E ? -1 : t0 < hd ? t0 : NU * E + t0;

    const void *src[5] = {a.y, a.res, per_row ? a.gate : nullptr, nullptr, nullptr};
    const int64_t ld[5] = {a.ld_y, a.ld_res, a.ld_gate, 0, 0};
    BlockRing ring{reinterpret_cast<uint64_t *>(smem), smem + BLOCK_HEADER + block_table_bytes(D), a.stages, a.stage_bytes, per_row ? 3 : 2};
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
    griddep_launch_dependents();
    if constexpr (KIND == BLOCK_STAGED) {
        if (threadIdx.x == 0)
            for (int s = 0; s < ring.S && s < deal.n; ++s) ring_issue<T>(ring, a, src, ld, deal.row(s), s, policy);
    }

    // A row's slots; the first row's loads go ahead of the weights' where no ring does.
    const int ry = KIND == BLOCK_WARP ? (int)(threadIdx.x >> 5) : 0;
    Raw vy[V], vr[V], vg[GROW ? V : 1];
    float xy = 0.f, xr = 0.f, xg = 1.f;  // of column cx
    auto fetch = [&](const T *py, const T *pr, const T *pg) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = SL::unit(j, t0, NT);
            if (u < NU) {
                vy[j] = SL::load(py, u, NT, NU);
                vr[j] = SL::load(pr, u, NT, NU);
                if constexpr (GROW) vg[j] = SL::load(pg, u, NT, NU);
            }
        }
        if constexpr (SHIFT)
            if (cx >= 0) {
                xy = Cvt<T>::load1(py + (cx - hd));
                xr = Cvt<T>::load1(pr + (cx - hd));
                if constexpr (GROW) xg = Cvt<T>::load1(pg + (cx - hd));
            }
    };
    auto fetch_global = [&](int64_t row) {
        fetch(static_cast<const T *>(a.y) + row * a.ld_y + hd, static_cast<const T *>(a.res) + row * a.ld_res + hd,
              per_row ? static_cast<const T *>(a.gate) + row * a.ld_gate + hd : nullptr);
    };
    if constexpr (KIND != BLOCK_STAGED)
        if (ry < deal.n) fetch_global(deal.row(ry));

    float *table = reinterpret_cast<float *>(smem + BLOCK_HEADER);
    Raw vw[KIND == BLOCK_STAGED ? 1 : V];
    float2 m[V][P];  // without the gate if it has a row for each row
    float xm = 0.f, xw = 0.f;  // m and w1 of column cx
    auto load_raw = [&](const void *base, int u) {  // of a row of weights or a gate row
        if constexpr (SHIFT) return SL::load_columns(static_cast<const T *>(base), hd + u * E);
        else return SL::load(base, u, NT, NU);
    };
    auto load_unit = [&](const void *base, int u, float2 (&f)[P]) { SL::unpack(load_raw(base, u), f); };
    auto load_m = [&](const T *gate_row) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = SL::unit(j, t0, NT);
            if (u < NU) {
                float2 f[P], q[P];
                if (post) load_unit(a.w_post, u, f);
                if (gate_row) load_unit(gate_row, u, q);
#pragma unroll
                for (int p = 0; p < P; ++p)
                    m[j][p] = f2mul(post ? f2add(both(a.weight_bias), f[p]) : both(1.f),
                                    gate_row ? f2mul(both(a.scale), q[p]) : both(a.scale));
            }
        }
        if constexpr (SHIFT)
            if (cx >= 0)
                xm = (post ? a.weight_bias + Cvt<T>::load1(static_cast<const T *>(a.w_post) + cx) : 1.f) *
                     (gate_row ? a.scale * Cvt<T>::load1(gate_row + cx) : a.scale);
    };
    if constexpr (SHIFT)
        if (cx >= 0) xw = a.weight_bias + Cvt<T>::load1(static_cast<const T *>(a.w_pre) + cx);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int u = SL::unit(j, t0, NT);
        if (u < NU) {
            const Raw w = load_raw(a.w_pre, u);
            if constexpr (KIND == BLOCK_STAGED) {  // a thread reads only what it wrote itself
                float2 f[P];
                SL::unpack(w, f);
#pragma unroll
                for (int p = 0; p < P; ++p) f[p] = f2add(both(a.weight_bias), f[p]);
                SL::put(table, u, NT, NU, f);
            } else {
                vw[j] = w;
            }
        }
    }
    if (!a.gate || per_row) load_m(nullptr);
    // w1 of slot j, first unit u
    auto w1_of = [&](int j, int u, float2 (&w)[P]) {
        if constexpr (KIND == BLOCK_STAGED) {
            SL::get(table, u, NT, NU, w);
        } else {
            SL::unpack(vw[j], w);
#pragma unroll
            for (int p = 0; p < P; ++p) w[p] = f2add(both(a.weight_bias), w[p]);
        }
    };


    int64_t group_end = a.gate && !per_row ? 0 : INT64_MAX;  // first row past the gate row held in m
    int s = 0;
    uint32_t ph = 0;
    for (int64_t ri = ry; ri < deal.n; ri += R) {
        const int64_t row = deal.row(ri);
        if (row >= group_end) {
            const int64_t gr = gate_row(row, a.rows_per_gate);
            group_end = (gr + 1) * a.rows_per_gate;
            load_m(static_cast<const T *>(a.gate) + gr * a.ld_gate);
        }
        bool ok = true;
        if constexpr (KIND == BLOCK_STAGED) {
            const unsigned char *st = ring.data + (size_t)s * ring.tensors * ring.stage_bytes;
            auto staged = [&](const void *base, int64_t ld) {
                const uintptr_t p = (uintptr_t)(static_cast<const T *>(base) + row * ld);
                const T *q = reinterpret_cast<const T *>(st + (p & 15u)) + hd;
                st += ring.stage_bytes;
                return q;
            };
            const T *py = staged(a.y, a.ld_y), *pr = staged(a.res, a.ld_res);
            const T *pg = per_row ? staged(a.gate, a.ld_gate) : nullptr;
            ok = mbar_wait_bounded(&ring.full[s], ph, a.wait_budget);
            fetch(py, pr, pg);
        }
        // v = m y of unit j, the added term before r_y
        auto added = [&](int j, const float2 (&y)[P], float2 (&v)[P]) {
#pragma unroll
            for (int p = 0; p < P; ++p) v[p] = f2mul(m[j][p], y[p]);
            if constexpr (GROW) {
                float2 q[P];
                SL::unpack(vg[j], q);
#pragma unroll
                for (int p = 0; p < P; ++p) v[p] = f2mul(v[p], q[p]);
            }
        };
        float2 s2[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};  // y^2, res^2, res v, v^2
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (SL::unit(j, t0, NT) < NU) {
                float2 y[P], r[P], v[P];
                SL::unpack(vy[j], y);
                SL::unpack(vr[j], r);
                added(j, y, v);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    s2[0] = f2fma(y[p], y[p], s2[0]);
                    s2[1] = f2fma(r[p], r[p], s2[1]);
                    s2[2] = f2fma(r[p], v[p], s2[2]);
                    s2[3] = f2fma(v[p], v[p], s2[3]);
                }
            }
        }
        const float xv = SHIFT ? xm * xy * (GROW ? xg : 1.f) : 0.f;  // v of column cx
        if constexpr (SHIFT)
            if (cx >= 0) {
                s2[0].x = fmaf(xy, xy, s2[0].x);
                s2[1].x = fmaf(xr, xr, s2[1].x);
                s2[2].x = fmaf(xr, xv, s2[2].x);
                s2[3].x = fmaf(xv, xv, s2[3].x);
            }
        float sum[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = s2[i].x + s2[i].y;
        if constexpr (KIND == BLOCK_WARP) {
            warp_sums<4>(sum);
        } else {
            ok = cta_sums<4, MAXW>(sum, s_red[ri & 1], nw, ok);
        }
        if constexpr (KIND == BLOCK_STAGED) {
            if (!ok) {  // leave once this CTA's copies have landed
                if (threadIdx.x == 0) {
                    atomicOr(a.status, DEVSTATUS_WAIT_TIMEOUT);
                    for (int64_t k = ri; k < deal.n && k < ri + ring.S; ++k)
                        if (deal.row(k) != a.drop_row)
                            mbar_wait_bounded(&ring.full[k % ring.S], (uint32_t)((k / ring.S) & 1), DEFAULT_WAIT_BUDGET);
                }
                return;
            }
            // every thread has its units of this stage in registers
            if (threadIdx.x == 0 && ri + ring.S < deal.n)
                ring_issue<T>(ring, a, src, ld, deal.row(ri + ring.S), s, policy);
        }
        if constexpr (MAXT * MINB > 512) {  // 96 registers or fewer
#pragma unroll
            for (int j = 0; j < V; ++j) {
                keep_packed(vy[j]);
                keep_packed(vr[j]);
            }
        }
        const float r_y = post ? rsqrtf(sum[0] * inv_D + a.eps) : 1.f;
        const float tail = r_y * r_y * sum[3];
        float ss = fmaf(2.f * r_y, sum[2], sum[1] + tail);
        // h of unit j
        auto joined = [&](int j, float2 (&h)[P]) {
            float2 y[P], r[P], v[P];
            SL::unpack(vy[j], y);
            SL::unpack(vr[j], r);
            added(j, y, v);
#pragma unroll
            for (int p = 0; p < P; ++p) h[p] = f2fma(v[p], both(r_y), r[p]);
        };
        // Also where v^2 left fp32's range on either side (below: the 2^-126 that a sum
        // of subnormals may be off by shows in the result).  The same in every thread
        // of the row.
        const float terms = sum[1] + tail;
        if (!(ss * 8.f >= terms && terms <= FLT_MAX) || r_y * r_y * 0x1p-100f > terms + (float)a.D * a.eps) {
            float2 t2 = both(0.f);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (SL::unit(j, t0, NT) < NU) {
                    float2 h[P];
                    joined(j, h);
#pragma unroll
                    for (int p = 0; p < P; ++p) t2 = f2fma(h[p], h[p], t2);
                }
            }
            if constexpr (SHIFT)
                if (cx >= 0) {
                    const float h = fmaf(xv, r_y, xr);
                    t2.x = fmaf(h, h, t2.x);
                }
            float one[1] = {t2.x + t2.y};
            if constexpr (KIND == BLOCK_WARP) {
                one[0] = group_sum<32>(one[0]);
            } else {
                __syncthreads();  // this row's sums have been read
                cta_sums<1, MAXW>(one, s_red[ri & 1], nw, true);
            }
            ss = one[0];
        }
        const float r_h = rsqrtf(ss * inv_D + a.eps);
        T *out = static_cast<T *>(a.out0) + row * a.ld_out0;
        T *nres = static_cast<T *>(a.out1) + row * a.ld_out1;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = SL::unit(j, t0, NT);
            if (u < NU) {
                float2 h[P];
                joined(j, h);
                float2 w[P];
                w1_of(j, u, w);
#pragma unroll
                for (int p = 0; p < P; ++p) w[p] = f2mul(f2mul(h[p], both(r_h)), w[p]);
                SL::store(nres + hd, u, NT, NU, h);
                SL::store(out + hd, u, NT, NU, w);
            }
        }
        if constexpr (SHIFT)
            if (cx >= 0) {
                const float h = fmaf(xv, r_y, xr);
                Cvt<T>::store1(nres + cx, h);
                Cvt<T>::store1(out + cx, h * r_h * xw);
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
        } else if constexpr (KIND == BLOCK_WARP) {
            if (ri + R < deal.n) fetch_global(deal.row(ri + R));
        }
    }
}

// VJP -----------------------------------------------------------------------
// FORM: which of a norm after the block, g_res and saved scales are there, known when
// compiled (FORM_ bits; 0: asked at run time).  HALF: 16 bytes of a row a thread
// instead of 32.
template <typename T, int UB, int MAXT, int MINB, int KIND, bool GROW, bool SHIFT, int FORM, bool HALF>
__global__ void __launch_bounds__(MAXT, MINB) block_vjp_kernel(const __grid_constant__ BlockArgs a) {
    using SL = Slot<T, UB>;
    using Raw = typename SL::Raw;
    constexpr int E = SL::E, V = HALF ? SL::COUNT / 2 : SL::COUNT, P = SL::P, MAXW = MAXT / 32;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float s_red[2][KIND == BLOCK_WARP ? 1 : MAXW][8];
    const int NT = KIND == BLOCK_WARP ? 32 : (int)blockDim.x;
    const int t0 = KIND == BLOCK_WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    const int R = KIND == BLOCK_WARP ? (int)(blockDim.x >> 5) : 1;
    const int ry = KIND == BLOCK_WARP ? (int)(threadIdx.x >> 5) : 0;
    const int D = a.D, nw = (int)(blockDim.x >> 5);
    const float inv_D = 1.0f / (float)D;
    constexpr bool per_row = GROW;  // a gate row for each row
    const bool post = FORM ? (FORM & FORM_POST) != 0 : a.w_post != nullptr;
    const bool more = FORM ? (FORM & FORM_MORE) != 0 : a.g_res != nullptr;
    const bool saved = FORM ? (FORM & FORM_SAVED) != 0 : a.rstd != nullptr;
    const int64_t cta = blockIdx.x;
    const RowDeal deal = vjp_rows(a, cta);
    // SHIFT: `hd` columns before a row's first 16-byte boundary, the same for all of
    // this CTA's rows; thread t0 also has column cx, one of those or of the rest behind
    // the last unit.
    const int hd = SHIFT ? (int)(-((uintptr_t)(static_cast<const T *>(a.y) + deal.row(0) * a.ld_y)) & 15u) / (int)sizeof(T) : 0;
    const int NU = SHIFT ? min((D - hd) / E, V * NT) : D / E;
    const int cx = !SHIFT || t0 >= D - NU * E ? -1 : t0 < hd ? t0 : NU * E + t0;

    const void *src[5] = {a.y, a.res, a.g, more ? a.g_res : nullptr, per_row ? a.gate : nullptr};
    const int64_t ld[5] = {a.ld_y, a.ld_res, a.ld_g, a.ld_g_res, a.ld_gate};
    BlockRing ring{reinterpret_cast<uint64_t *>(smem), smem + BLOCK_HEADER + block_table_bytes(D), a.stages, a.stage_bytes,
                   3 + more + per_row};
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
    griddep_launch_dependents();
    if constexpr (KIND == BLOCK_STAGED) {
        if (threadIdx.x == 0)
            for (int s = 0; s < ring.S && s < deal.n; ++s) ring_issue<T>(ring, a, src, ld, deal.row(s), s, policy);
    }

    // A row's slots; the first row's loads go ahead of the weights' where no ring does.
    Raw vy[V], vh[V], vg[V], vr[V], va[GROW ? V : 1];
    float xy = 0.f, xh = 0.f, xg = 0.f, xr = 0.f, xa = 1.f;  // of column cx
    auto fetch = [&](const T *py, const T *ph, const T *pg, const T *pr, const T *pa) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = SL::unit(j, t0, NT);
            if (u < NU) {
                vy[j] = SL::load(py, u, NT, NU);
                vh[j] = SL::load(ph, u, NT, NU);
                vg[j] = SL::load(pg, u, NT, NU);
                if (more) vr[j] = SL::load(pr, u, NT, NU);
                if constexpr (GROW) va[j] = SL::load(pa, u, NT, NU);
            }
        }
        if constexpr (SHIFT)
            if (cx >= 0) {
                xy = Cvt<T>::load1(py + (cx - hd));
                xh = Cvt<T>::load1(ph + (cx - hd));
                xg = Cvt<T>::load1(pg + (cx - hd));
                if (more) xr = Cvt<T>::load1(pr + (cx - hd));
                if constexpr (GROW) xa = Cvt<T>::load1(pa + (cx - hd));
            }
    };
    auto fetch_global = [&](int64_t row) {
        fetch(static_cast<const T *>(a.y) + row * a.ld_y + hd, static_cast<const T *>(a.res) + row * a.ld_res + hd,
              static_cast<const T *>(a.g) + row * a.ld_g + hd,
              more ? static_cast<const T *>(a.g_res) + row * a.ld_g_res + hd : nullptr,
              per_row ? static_cast<const T *>(a.gate) + row * a.ld_gate + hd : nullptr);
    };
    if constexpr (KIND != BLOCK_STAGED)
        if (ry < deal.n) fetch_global(deal.row(ry));
    int64_t fetched = ry;  // the row in the slots

    float *table = reinterpret_cast<float *>(smem + BLOCK_HEADER);
    Raw vw[KIND == BLOCK_STAGED ? 1 : V];
    float2 m[V][P], acc_pre[V][P], acc_mid[V][P];
    float xm = 0.f, xw = 0.f, x_pre = 0.f, x_mid = 0.f;  // of column cx
    auto load_raw = [&](const void *base, int u) {  // of a row of weights or a gate row
        if constexpr (SHIFT) return SL::load_columns(static_cast<const T *>(base), hd + u * E);
        else return SL::load(base, u, NT, NU);
    };
    auto load_unit = [&](const void *base, int u, float2 (&f)[P]) { SL::unpack(load_raw(base, u), f); };
    auto load_m = [&](const T *gate_row) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int u = SL::unit(j, t0, NT);
            if (u < NU) {
                float2 f[P], q[P];
                if (post) load_unit(a.w_post, u, f);
                if (gate_row) load_unit(gate_row, u, q);
#pragma unroll
                for (int p = 0; p < P; ++p)
                    m[j][p] = f2mul(post ? f2add(both(a.weight_bias), f[p]) : both(1.f),
                                    gate_row ? f2mul(both(a.scale), q[p]) : both(a.scale));
            }
        }
        if constexpr (SHIFT)
            if (cx >= 0)
                xm = (post ? a.weight_bias + Cvt<T>::load1(static_cast<const T *>(a.w_post) + cx) : 1.f) *
                     (gate_row ? a.scale * Cvt<T>::load1(gate_row + cx) : a.scale);
    };
    if constexpr (SHIFT)
        if (cx >= 0) xw = a.weight_bias + Cvt<T>::load1(static_cast<const T *>(a.w_pre) + cx);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int u = SL::unit(j, t0, NT);
        if (u < NU) {
            const Raw w = load_raw(a.w_pre, u);
            if constexpr (KIND == BLOCK_STAGED) {  // a thread reads only what it wrote itself
                float2 f[P];
                SL::unpack(w, f);
#pragma unroll
                for (int p = 0; p < P; ++p) f[p] = f2add(both(a.weight_bias), f[p]);
                SL::put(table, u, NT, NU, f);
            } else {
                vw[j] = w;
            }
        }
#pragma unroll
        for (int p = 0; p < P; ++p) acc_pre[j][p] = acc_mid[j][p] = both(0.f);
    }
    if (!a.gate || per_row) load_m(nullptr);
    // w1 of slot j, first unit u
    auto w1_of = [&](int j, int u, float2 (&w)[P]) {
        if constexpr (KIND == BLOCK_STAGED) {
            SL::get(table, u, NT, NU, w);
        } else {
            SL::unpack(vw[j], w);
#pragma unroll
            for (int p = 0; p < P; ++p) w[p] = f2add(both(a.weight_bias), w[p]);
        }
    };

    auto store_floats = [&](float *row, int u, const float2 (&f)[P], float k) {
        if constexpr (SHIFT) SL::store_floats_at(row, hd + u * E, f, k);
        else SL::store_floats(row, u, NT, NU, f, k);
    };
    // Writes k times the accumulators to the row dst (BLOCK_WARP: the warps' added
    // in warp order) and clears them.
    auto flush = [&](float2 (&acc)[V][P], float &extra, float *dst, float k) {
        if (KIND == BLOCK_WARP && R > 1) {
            float *buf = reinterpret_cast<float *>(smem);  // [R][D]
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int u = SL::unit(j, t0, NT);
                if (u < NU) SL::store_floats(buf + (size_t)ry * (block_sum_bytes(D) / 4), u, NT, NU, acc[j], k);
            }
            __syncthreads();
            for (int c = threadIdx.x; c < D; c += blockDim.x) {
                float t = buf[c];
                for (int w = 1; w < R; ++w) t += buf[(size_t)w * (block_sum_bytes(D) / 4) + c];
                dst[c] = t;
            }
            __syncthreads();  // buf may be written again
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int u = SL::unit(j, t0, NT);
                if (u < NU) store_floats(dst, u, acc[j], k);
            }
            if constexpr (SHIFT)
                if (cx >= 0) dst[cx] = extra * k;
            extra = 0.f;
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int p = 0; p < P; ++p) acc[j][p] = both(0.f);
    };

    // a.cluster: this CTA's sums, of gw_pre and of A, behind the warps' rows
    auto sums_of = [&](int i) {
        const size_t row = block_sum_bytes(D) / 4;
        return reinterpret_cast<float *>(smem) + (KIND == BLOCK_WARP ? R + i : i) * row;
    };

    int s = 0;
    uint32_t ph = 0;
    for (int64_t seg = 0; seg < deal.n;) {  // rows of one gate row: deal.row(seg), ..., deal.row(end - 1)
        const int64_t gr = per_row ? 0 : gate_row(deal.row(seg), a.rows_per_gate);
        const int64_t end = per_row || a.team ? deal.n : min(deal.n, (gr + 1) * a.rows_per_gate - deal.lo);
        if (a.gate && !per_row) load_m(static_cast<const T *>(a.gate) + gr * a.ld_gate);
        for (int64_t ri = seg + ry; ri < end; ri += R) {
            const int64_t row = deal.row(ri);
            float r_y = 1.f, r_h = 0.f;
            if (saved) {
                if (post) r_y = __ldg(a.rstd + row);
                r_h = __ldg(a.rstd + a.rows + row);
            }
            bool ok = true;
            if constexpr (KIND == BLOCK_STAGED) {
                const unsigned char *st = ring.data + (size_t)s * ring.tensors * ring.stage_bytes;
                auto staged = [&](const void *base, int64_t ld) {
                    const uintptr_t p = (uintptr_t)(static_cast<const T *>(base) + row * ld);
                    const T *q = reinterpret_cast<const T *>(st + (p & 15u)) + hd;
                    st += ring.stage_bytes;
                    return q;
                };
                const T *py = staged(a.y, a.ld_y), *phh = staged(a.res, a.ld_res), *pgo = staged(a.g, a.ld_g);
                const T *pgr = more ? staged(a.g_res, a.ld_g_res) : nullptr;
                const T *pga = per_row ? staged(a.gate, a.ld_gate) : nullptr;
                ok = mbar_wait_bounded(&ring.full[s], ph, a.wait_budget);
                fetch(py, phh, pgo, pgr, pga);
            } else if (ri != fetched) {
                fetch_global(row);
            }
            // m of unit j with the row's own gate
            auto mult = [&](int j, float2 (&mm)[P]) {
#pragma unroll
                for (int p = 0; p < P; ++p) mm[p] = m[j][p];
                if constexpr (GROW) {
                    float2 q[P];
                    SL::unpack(va[j], q);
#pragma unroll
                    for (int p = 0; p < P; ++p) mm[p] = f2mul(mm[p], q[p]);
                }
            };
            // a h, u a, u h, u g_res (a = g w1, u = m y), h^2, y^2
            float2 s2[6] = {both(0.f), both(0.f), both(0.f), both(0.f), both(0.f), both(0.f)};
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (SL::unit(j, t0, NT) < NU) {
                    float2 y[P], h[P], x[P], u[P], w[P];
                    SL::unpack(vy[j], y);
                    SL::unpack(vh[j], h);
                    SL::unpack(vg[j], x);
                    mult(j, u);
                    w1_of(j, SL::unit(j, t0, NT), w);
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        x[p] = f2mul(x[p], w[p]);
                        u[p] = f2mul(u[p], y[p]);
                        s2[0] = f2fma(x[p], h[p], s2[0]);
                        s2[1] = f2fma(u[p], x[p], s2[1]);
                        s2[2] = f2fma(u[p], h[p], s2[2]);
                    }
                    if (more) {
                        SL::unpack(vr[j], x);
#pragma unroll
                        for (int p = 0; p < P; ++p) s2[3] = f2fma(u[p], x[p], s2[3]);
                    }
                    if (!saved) {
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            s2[4] = f2fma(h[p], h[p], s2[4]);
                            s2[5] = f2fma(y[p], y[p], s2[5]);
                        }
                    }
                }
            }
            if constexpr (SHIFT)
                if (cx >= 0) {
                    const float x = xg * xw, u = xm * (GROW ? xa : 1.f) * xy;
                    s2[0].x = fmaf(x, xh, s2[0].x);
                    s2[1].x = fmaf(u, x, s2[1].x);
                    s2[2].x = fmaf(u, xh, s2[2].x);
                    s2[3].x = fmaf(u, xr, s2[3].x);
                    if (!saved) {
                        s2[4].x = fmaf(xh, xh, s2[4].x);
                        s2[5].x = fmaf(xy, xy, s2[5].x);
                    }
                }
            float sum[6];
#pragma unroll
            for (int i = 0; i < 6; ++i) sum[i] = s2[i].x + s2[i].y;
            if constexpr (KIND == BLOCK_WARP) {
                if (saved) warp_sums<4>(reinterpret_cast<float (&)[4]>(sum));
                else warp_sums<6>(sum);
            } else {
                ok = saved ? cta_sums<4, MAXW>(reinterpret_cast<float (&)[4]>(sum), s_red[ri & 1], nw, ok)
                           : cta_sums<6, MAXW>(sum, s_red[ri & 1], nw, ok);
            }
            if constexpr (KIND == BLOCK_STAGED) {
                if (!ok) {
                    if (threadIdx.x == 0) {
                        atomicOr(a.status, DEVSTATUS_WAIT_TIMEOUT);
                        for (int64_t k = ri; k < deal.n && k < ri + ring.S; ++k)
                            if (deal.row(k) != a.drop_row)
                                mbar_wait_bounded(&ring.full[k % ring.S], (uint32_t)((k / ring.S) & 1),
                                                  DEFAULT_WAIT_BUDGET);
                    }
                    return;
                }
                // every thread has its slots of this stage in registers
                if (threadIdx.x == 0 && ri + ring.S < deal.n)
                    ring_issue<T>(ring, a, src, ld, deal.row(ri + ring.S), s, policy);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                keep_packed(vy[j]);
                keep_packed(vh[j]);
                keep_packed(vg[j]);
                keep_packed(vr[j]);
            }
            if (!saved) {
                r_h = rsqrtf(sum[4] * inv_D + a.eps);
                if (post) r_y = rsqrtf(sum[5] * inv_D + a.eps);
            }
            // scale by scale: without an epsilon a tiny row's r^2 can leave fp32's range
            const float cc = r_h * (r_h * (sum[0] * inv_D));
            const float dot = fmaf(r_h, sum[1] - cc * sum[2], sum[3]);  // sum of m g_h y
            const float ee = post ? r_y * (r_y * (dot * inv_D)) : 0.f;
            T *gy = static_cast<T *>(a.out0) + row * a.ld_out0;
            T *gh = static_cast<T *>(a.out1) + row * a.ld_out1;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int u = SL::unit(j, t0, NT);
                if (u < NU) {
                    float2 h[P], x[P], z[P], w[P];
                    w1_of(j, u, w);
                    SL::unpack(vh[j], h);
                    SL::unpack(vg[j], x);
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        acc_pre[j][p] = f2fma(x[p], f2mul(h[p], both(r_h)), acc_pre[j][p]);
                        z[p] = f2mul(f2fma(h[p], both(-cc), f2mul(x[p], w[p])), both(r_h));
                    }
                    if (more) {
                        SL::unpack(vr[j], x);
#pragma unroll
                        for (int p = 0; p < P; ++p) z[p] = f2add(z[p], x[p]);
                    }
                    SL::store(gh + hd, u, NT, NU, z);  // g_h
                    float2 y[P], mm[P];
                    SL::unpack(vy[j], y);
                    mult(j, mm);
#pragma unroll
                    for (int p = 0; p < P; ++p) h[p] = f2mul(z[p], f2mul(y[p], both(r_y)));  // g_h y r_y
                    if constexpr (GROW) {  // this row is its gate row: finished here, and gw_post's term weighted
                        float2 w2[P];
                        SL::unpack(va[j], x);
                        if (post) load_unit(a.w_post, u, w2);
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            acc_mid[j][p] = f2fma(h[p], x[p], acc_mid[j][p]);
                            w2[p] = f2mul(h[p], post ? f2add(both(a.weight_bias), w2[p]) : both(1.f));
                        }
                        store_floats(a.g_gate + row * D, u, w2, a.scale);
                    } else {
#pragma unroll
                        for (int p = 0; p < P; ++p) acc_mid[j][p] = f2add(h[p], acc_mid[j][p]);
                    }
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        z[p] = f2mul(f2fma(y[p], both(-ee), f2mul(mm[p], z[p])), both(r_y));
                    SL::store(gy + hd, u, NT, NU, z);
                }
            }
            if constexpr (SHIFT)
                if (cx >= 0) {
                    x_pre = fmaf(xg, xh * r_h, x_pre);
                    const float z = r_h * fmaf(xh, -cc, xg * xw) + xr, q = z * (xy * r_y);
                    Cvt<T>::store1(gh + cx, z);
                    if constexpr (GROW) {
                        x_mid = fmaf(q, xa, x_mid);
                        const float w2 = post ? a.weight_bias + Cvt<T>::load1(static_cast<const T *>(a.w_post) + cx) : 1.f;
                        a.g_gate[row * D + cx] = q * w2 * a.scale;
                    } else {
                        x_mid += q;
                    }
                    Cvt<T>::store1(gy + cx, r_y * fmaf(xy, -ee, xm * (GROW ? xa : 1.f) * z));
                }
            if constexpr (KIND == BLOCK_STAGED) {
                if (++s == ring.S) {
                    s = 0;
                    ph ^= 1u;
                }
            } else if constexpr (KIND == BLOCK_WARP) {
                // the next gate row's rows are dealt out to the warps from its first on
                fetched = ri + R < end ? ri + R : end + ry;
                if (fetched < deal.n) fetch_global(deal.row(fetched));
            }
        }
        if (KIND != BLOCK_STAGED && a.cluster) {
            if (a.gate || post) flush(acc_mid, x_mid, sums_of(1), a.scale);  // the only segment
        } else if (a.gate || post) {
            const bool whole = a.g_gate && !per_row && end - seg == a.rows_per_gate;
            flush(acc_mid, x_mid,
                  per_row ? a.part_mid + 2 * cta * D
                  : whole ? a.g_gate + gr * D
                          : a.part_mid + mid_slot(cta, seg == 0) * D,
                  a.scale);
        }
        seg = end;
    }
    if constexpr (KIND != BLOCK_STAGED)
        if (a.cluster) {
            // The second stage, here: each CTA takes columns and adds up all CTAs' sums of
            // them in the CTAs' order, gate row by gate row (several only with a row a CTA).
            flush(acc_pre, x_pre, sums_of(0), 1.f);
            cluster_sync_all();
            const int ctas = a.cluster, rpg = (int)min(a.rows_per_gate, (int64_t)16);
            for (int c = (int)cta * (int)blockDim.x + (int)threadIdx.x; c < D; c += ctas * (int)blockDim.x) {
                float v[2][8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < ctas) {
                        v[0][r] = load_remote(sums_of(0) + c, r);
                        if (a.gate || post) v[1][r] = load_remote(sums_of(1) + c, r);
                    }
                float pre = 0.f, A = 0.f, gp = 0.f;
                const float w2 = post ? a.weight_bias + Cvt<T>::load1(static_cast<const T *>(a.w_post) + c) : 1.f;
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < ctas) {
                        pre += v[0][r];
                        if (a.gate || post) A += v[1][r];
                        const bool last = r == ctas - 1 || (!per_row && (r + 1) % rpg == 0);
                        if (last) {
                            float k = 1.f;
                            if (a.gate && !per_row) {
                                k = Cvt<T>::load1(static_cast<const T *>(a.gate) + (int64_t)(r / rpg) * a.ld_gate + c);
                                a.g_gate[(int64_t)(r / rpg) * D + c] = A * w2;
                            }
                            gp = fmaf(k, A, gp);
                            A = 0.f;
                        }
                    }
                a.gw_pre[c] = pre;
                if (post) a.gw_post[c] = gp;
            }
            cluster_sync_all();  // no CTA leaves while another reads its sums
            return;
        }
    flush(acc_pre, x_pre, a.part_pre + cta * D, 1.f);
}

}  // namespace rmsn
