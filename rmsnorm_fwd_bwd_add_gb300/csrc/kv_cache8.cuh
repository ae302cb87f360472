// kv_cache8.cuh -- kernels of the 8-bit cache: the append that rotates, quantises and
// writes a step's tokens, and the read that brings them back.
//
// A head x (of k, rotated and unrounded, or of v) has a = max(max |x|, top 2^-126), scale =
// a / top and codes round(x top / a), top = 448 (e4m3) or 127 (int8); it is read back as code *
// scale.  Both directions are bound by memory: q, k and v are read once, q_out, codes and
// scales written once.
//
// On the GB300 (6.8 TB/s copied), inputs changing from call to call: 16384 tokens of 32 + 8
// heads of 128 (bf16, three axes, e4m3) appended in 60 us (91 % of that), 8 tokens in 3.8 us
// (two trips to memory and the cosines); 65536 tokens of 8 heads of 128 read in 65 us (92 %),
// 77 in 2.1 us.
#pragma once

#include "quant.cuh"
#include "rope_ex.cuh"

namespace rmsn {

constexpr int C8_NT = 256;

// [num_slots, Hkv] scales: strides in elements.
struct Scales {
    float *p;
    int64_t st, sh;
};

struct AppendArgs : RopeArgs<true> {
    Scales k_scale, v_scale;
};

// Codes of VE elements as one word.
template <int VE> struct CodeWord;
template <> struct CodeWord<8> { using type = uint2; };
template <> struct CodeWord<4> { using type = uint32_t; };
template <> struct CodeWord<2> { using type = uint16_t; };
template <> struct CodeWord<1> { using type = uint8_t; };

template <int FMT, int VE> __device__ __forceinline__ typename CodeWord<VE>::type code_word(const float (&f)[VE], float2 by) {
    if constexpr (VE >= 4) {
        uint32_t c[VE / 4];
#pragma unroll
        for (int i = 0; i < VE / 4; ++i) {
            const float2 x = in_codes(make_float2(f[4 * i], f[4 * i + 1]), by);
            const float2 y = in_codes(make_float2(f[4 * i + 2], f[4 * i + 3]), by);
            c[i] = code_quad<FMT>(x.x, x.y, y.x, y.y);
        }
        if constexpr (VE == 8) return make_uint2(c[0], c[1]);
        else return c[0];
    } else {
        return (typename CodeWord<VE>::type)code_pair<FMT>(in_codes(f[0], by), VE == 2 ? in_codes(f[VE - 1], by) : 0.f);
    }
}

template <typename T, int VB, int VE> __device__ __forceinline__ void unpack_raw(const typename RawUnit<VB>::type &v, float (&f)[VE]) {
    if constexpr (VE == 2) {
        const float2 p = Cvt<T>::unpack2(v);
        f[0] = p.x;
        f[1] = p.y;
    } else {
        unpack_unit<T, VB>(v, f);
    }
}
template <typename T, int VB, int VE> __device__ __forceinline__ typename RawUnit<VB>::type pack_raw(const float (&f)[VE]) {
    if constexpr (VE == 2) return Cvt<T>::pack2(f[0], f[1]);
    else return pack_unit<T, VB>(f);
}

// VE floats from shared memory, at a multiple of their number.
template <int VE> __device__ __forceinline__ void load_floats(const float *p, float (&f)[VE]) {
    if constexpr (VE >= 4) {
#pragma unroll
        for (int i = 0; i < VE / 4; ++i) {
            const float4 v = reinterpret_cast<const float4 *>(p)[i];
            f[4 * i] = v.x;
            f[4 * i + 1] = v.y;
            f[4 * i + 2] = v.z;
            f[4 * i + 3] = v.w;
        }
    } else if constexpr (VE == 2) {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        f[0] = v.x;
        f[1] = v.y;
    } else {
        f[0] = p[0];
    }
}

constexpr int C8_CTAS_PER_SM = 2;

// Hides from the compiler that a register's value is unchanged, so that it is unpacked
// again instead of being held unpacked.
__device__ __forceinline__ void same_bits(uint4 &v) { asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)); }
__device__ __forceinline__ void same_bits(uint32_t &v) { asm volatile("" : "+r"(v)); }
__device__ __forceinline__ void same_bits(uint16_t &v) { asm volatile("" : "+h"(v)); }

// Smaller units come as whole heads in the 16-byte words of memory: the bytes that a head
// of `bytes` may touch.
__host__ __device__ constexpr int append8_head_bytes(int bytes) { return (bytes + 30) / 16 * 16; }

// A step's copies in shared memory, and the steps that a warp's ring holds: 3 KB of them,
// or 2 where as much is written as read.  Reading further ahead holds up the writes (16384
// tokens of 32 + 8 heads of 128: the 8-bit append 60.0 us, 61.9 with 2 KB, 65.1 with 4,
// 67.9 with 6, with three CTAs an SM 79; the rotation alone 53.6 with 2 KB, 58.6 with 3,
// 59.5 with 4).
template <int VB, int UPL> __host__ __device__ inline int append8_step_bytes(int head_bytes, int cw) {
    return VB == 16 ? 2 * UPL * 32 * VB : 32 / cw * append8_head_bytes(head_bytes);
}
template <int VB, int UPL, int FMT> __host__ __device__ constexpr int append8_ring() {
    constexpr int n = VB == 16 ? (FMT == RMSNORM_CACHE_SAME ? 2 : 3) * 1024 / (2 * UPL * 32 * VB) : 4;
    return n < 2 ? 2 : n;
}

__device__ __forceinline__ void copy_async16(unsigned char *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}

// Shared memory of a warp: the cosines, then the sines of a token's pairs; and its ring.
__host__ __device__ constexpr int append8_plane(int rot) { return (rot / 2 + 3) / 4 * 4; }

// FMT is RMSNORM_CACHE_SAME for caches of the inputs' type and, without slots, for
// rmsnorm_rope_axes, whose k stays with its token (VB = 16 alone).
//
// A warp takes a token (or one of a token's `wpt` parts, from token `whole` on), 32 / cw
// heads a step: cw lanes a head, UPL units of two vectors each a lane (rope_ex.cuh's
// units), so that a head's largest value is a few shuffles away.  The token's cosines and
// sines are computed by the warp's lanes together, once for all of its heads.
//
// A lane copies its vectors of the steps to come, through all of its tokens, into a ring
// of its own in shared memory: with two batches of steps in registers instead a warp
// waited for memory five times a token (16384 tokens of 32 + 8 heads of 128: 70 us, 60
// so).  Heads in smaller units (off 16-byte boundaries, or turned by an odd number of
// pairs) are copied whole, in the words of memory, which the head's lanes share.
template <typename T, int VB, bool INTERLEAVED, int FMT, int UPL>
__global__ void __launch_bounds__(C8_NT, C8_CTAS_PER_SM) append8_kernel(const __grid_constant__ AppendArgs a, int64_t whole, int wpt, int cw) {
    using V = typename RawUnit<VB>::type;
    constexpr int VE = VB / (int)sizeof(T), RING = append8_ring<VB, UPL, FMT>();
    constexpr bool PAIRED = INTERLEAVED && VE > 1;
    using Codes = typename CodeWord<VE>::type;
    constexpr bool SAME = FMT == RMSNORM_CACHE_SAME;
    extern __shared__ __align__(16) unsigned char s_dyn[];
    const int lane = threadIdx.x & 31, half = a.rot / 2, plane = append8_plane(a.rot);
    constexpr bool WORDS = VB < 16;
    const int STEP = append8_step_bytes<VB, UPL>(a.Dh * (int)sizeof(T), cw);
    unsigned char *s_ring = s_dyn + (threadIdx.x >> 5) * RING * STEP;
    float *s_cos = reinterpret_cast<float *>(s_dyn + (C8_NT / 32) * RING * STEP) + (threadIdx.x >> 5) * 2 * plane;
    float *s_sin = s_cos + plane;
    __shared__ float2 s_turns[RX_MAX_DH / 2];
    __shared__ uint8_t s_axis[RX_MAX_DH / 2];
    for (int i = threadIdx.x; i < half; i += C8_NT) {
        s_turns[i] = a.turns[i];
        s_axis[i] = a.axes.of[i];
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();

    const int hpi = 32 / cw, hs = lane / cw, lu = lane - hs * cw;
    const HeadMap<VE, PAIRED, INTERLEAVED> map(a.Dh, a.rot), v_map(a.Dh, 0);
    // unit i of this lane: first elements of its two vectors in a head of q or k, and of v
    int ia[UPL], ib[UPL], va[UPL], vb[UPL];
    uint32_t in = 0, two = 0, turns = 0, v_in = 0, v_two = 0;  // a bit a unit
#pragma unroll
    for (int i = 0; i < UPL; ++i) {
        const int l = lu + i * cw;
        bool w;
        map.at(l, ia[i], ib[i], w);
        if (hs < hpi && l < map.lanes) in |= 1u << i, two |= (uint32_t)w << i;
        if (l < map.rot_units) turns |= 1u << i;
        v_map.at(l, va[i], vb[i], w);
        if (hs < hpi && l < v_map.lanes) v_in |= 1u << i, v_two |= (uint32_t)w << i;
    }
    turns &= in;
    // this lane's vectors of a step, or its head's words
    s_ring += WORDS ? (hs < hpi ? hs : 0) * append8_head_bytes(a.Dh * (int)sizeof(T)) : lane * VB;
    const uint32_t q_in = a.q_out.p != a.q.p ? in : turns;  // in place: nothing to copy
    const uint32_t k_in = !SAME || a.k_out.p != a.k.p ? in : turns;
    const int kinds = a.slots ? 3 : 2;
    // A token's place in q, k, v or q_out, in elements.
    auto place = [&](const Heads &x, int64_t t) {
        if (!SAME || a.S == a.T) return t * x.st;
        const int64_t b = t / a.S;
        return b * x.sb + (t - b * a.S) * x.st;
    };
    // the largest of a head's cw lanes: butterflies, or turns of 1, 2, 4, ... lanes around
    // them (counting some twice does no harm)
    const bool square = (cw & (cw - 1)) == 0;
    auto head_max = [&](float top) {
        if (square) return run_max(top, cw);
        for (int off = 1; off < cw; off *= 2) {
            const int at = lu + off;
            top = max_abs(top, __shfl_sync(0xffffffffu, top, hs < hpi ? lane - lu + (at < cw ? at : at - cw) : lane));
        }
        return top;
    };
    const int64_t n_items = whole + (a.T - whole) * wpt, n_warps = (int64_t)gridDim.x * (C8_NT / 32);
    const int wshift = 31 - __clz(wpt);  // wpt is a power of two
    int64_t w = ((int64_t)blockIdx.x * C8_NT + threadIdx.x) >> 5;
    auto token_of = [&](int64_t item) { return item < whole ? item : whole + ((item - whole) >> wshift); };
    auto part_of = [&](int64_t item) { return item < whole ? 0 : (int)((item - whole) & (wpt - 1)); };
    auto parts_of = [&](int64_t item) { return item < whole ? 1 : wpt; };
    // The copies run ahead through the items, the kinds 0 (q), 1 (k) and 2 (v) of each and
    // the steps of a kind: this lane's next head and its address.
    int64_t ahead = w;
    int ahead_kind = 0, ahead_h = 0, ahead_heads = 0, ahead_at = 0, ahead_step = 0;
    const unsigned char *ahead_src = nullptr;
    auto begin_kind = [&] {
        const Heads &x = ahead_kind == 0 ? a.q : ahead_kind == 1 ? a.k : a.v;
        ahead_heads = ahead_kind == 0 ? a.Hq : a.Hkv;
        ahead_h = part_of(ahead) * hpi + hs;
        ahead_step = parts_of(ahead) * hpi;
        ahead_src = (const unsigned char *)x.p + (place(x, token_of(ahead)) * (int64_t)sizeof(T) + (uint64_t)(uint32_t)ahead_h * x.head_bytes);
    };
    auto first_kind = [&] {  // from ahead_kind on, that has heads in this part
        while (ahead < n_items) {
            begin_kind();
            if (ahead_h - hs < ahead_heads) return;
            if (++ahead_kind == kinds) {
                ahead_kind = 0;
                ahead += n_warps;
            }
        }
    };
    auto copy_ahead = [&] {
        if (ahead < n_items) {
            const bool is_v = ahead_kind == 2;
            unsigned char *dst = s_ring + ahead_at * STEP;
            if (ahead_h < ahead_heads) {
                if constexpr (WORDS) {
                    const unsigned char *from = (const unsigned char *)((uintptr_t)ahead_src & ~(uintptr_t)15);
                    const int end = (int)(ahead_src - from) + a.Dh * (int)sizeof(T);
                    if (hs < hpi)
                        for (int b = lu * 16; b < end; b += cw * 16) copy_async16(dst + b, from + b);
                } else {
                    const uint32_t wanted = ahead_kind == 0 ? q_in : is_v ? v_in : k_in, both = wanted & (is_v ? v_two : two);
                    const T *src = reinterpret_cast<const T *>(ahead_src);
#pragma unroll
                    for (int i = 0; i < UPL; ++i) {
                        if (wanted >> i & 1) copy_async16(dst + 2 * i * 32 * VB, src + (is_v ? va[i] : ia[i]));
                        if (both >> i & 1) copy_async16(dst + (2 * i + 1) * 32 * VB, src + (is_v ? vb[i] : ib[i]));
                    }
                }
            }
            ahead_h += ahead_step;
            ahead_src += (uint64_t)(uint32_t)ahead_step * (ahead_kind == 0 ? a.q.head_bytes : is_v ? a.v.head_bytes : a.k.head_bytes);
            if (ahead_h - hs >= ahead_heads) {
                if (++ahead_kind == kinds) {
                    ahead_kind = 0;
                    ahead += n_warps;
                }
                first_kind();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ahead_at = ahead_at + 1 == RING ? 0 : ahead_at + 1;
    };
    first_kind();
    int64_t p_next = 0, slot_next = 0;  // of the item ahead; lane x has its position on axis x
    auto look_ahead = [&](int64_t t) {
        slot_next = SAME && !a.slots ? 0 : a.slots[t];
        if (lane < a.axes.n) p_next = a.positions[lane * a.T + t];
    };
    if (w < n_items) look_ahead(token_of(w));
    for (int i = 0; i < RING; ++i) copy_ahead();
    int at = 0;  // place of the next step in the ring
    for (; w < n_items; w += n_warps) {
        const int64_t t = token_of(w), slot = slot_next;
        const int part = part_of(w), h_step = parts_of(w) * hpi;  // from a lane's head to its next
        const float2 mine = split_position(p_next);
        const bool pos_ok = __all_sync(0xffffffffu, p_next >= 0);
        if (w + n_warps < n_items) look_ahead(token_of(w + n_warps));
        const bool slot_ok = slot < a.num_slots, kept = slot_ok && slot >= 0;
        if ((!pos_ok || !slot_ok) && lane == 0 && part == 0) atomicOr(a.status, BAD_INDEX);
        __syncwarp();  // the token before has been read
        for (int m0 = 0; m0 < half; m0 += 32) {
            const int m = min(m0 + lane, half - 1), axis = s_axis[m];
            const float2 p = make_float2(__shfl_sync(0xffffffffu, mine.x, axis), __shfl_sync(0xffffffffu, mine.y, axis));
            const float2 c = cos_sin<!SAME || sizeof(T) == 4>(p, s_turns[m]);
            s_cos[m] = c.x * a.scale;
            s_sin[m] = c.y * (a.scale * a.sign);
        }
        __syncwarp();
        // Unit i of a head turned.  (Its cosines and sines come from shared memory each
        // time: 16 registers for whole vectors.)
        auto turn = [&](int i, float (&fa)[VE], float (&fb)[VE]) {
            if constexpr (PAIRED) {
                auto pairs = [&](float (&f)[VE], int from) {
                    float cs[VE / 2], sn[VE / 2];
                    load_floats(s_cos + from / 2, cs);
                    load_floats(s_sin + from / 2, sn);
#pragma unroll
                    for (int m = 0; m < VE / 2; ++m) {
                        const float x = f[2 * m], y = f[2 * m + 1];
                        f[2 * m] = fmaf(-y, sn[m], x * cs[m]);
                        f[2 * m + 1] = fmaf(x, sn[m], y * cs[m]);
                    }
                };
                pairs(fa, ia[i]);
                if (two >> i & 1) pairs(fb, ib[i]);
            } else {
                float cs[VE], sn[VE];
                const int first = VE == 1 && INTERLEAVED ? ia[i] / 2 : ia[i];
                load_floats(s_cos + first, cs);
                load_floats(s_sin + first, sn);
                if constexpr (VE > 1) {
#pragma unroll
                    for (int m = 0; m < VE; m += 2) {
                        const float2 x = make_float2(fa[m], fa[m + 1]), y = make_float2(fb[m], fb[m + 1]);
                        const float2 c = make_float2(cs[m], cs[m + 1]), s = make_float2(sn[m], sn[m + 1]);
                        const float2 xc = f2mul(x, c), yc = f2fma(x, s, f2mul(y, c));
                        fa[m] = fmaf(-y.x, s.x, xc.x);
                        fa[m + 1] = fmaf(-y.y, s.y, xc.y);
                        fb[m] = yc.x;
                        fb[m + 1] = yc.y;
                    }
                } else {
                    const float x = fa[0], y = fb[0];
                    fa[0] = fmaf(-y, sn[0], x * cs[0]);
                    fb[0] = fmaf(x, sn[0], y * cs[0]);
                }
            }
        };
        // The steps of one kind, in a loop that all lanes run: f(xa, xb, h) has a head's units.
        auto steps = [&](const Heads &x, int n, uint32_t wanted, uint32_t both, const int (&at_a)[UPL], const int (&at_b)[UPL], auto f) {
            for (int h = part * hpi + hs; h - hs < n; h += h_step) {
                V xa[UPL], xb[UPL];
                asm volatile("cp.async.wait_group %0;" ::"n"(RING - 1) : "memory");
                if constexpr (WORDS) {
                    __syncwarp();  // the other lanes' copies too
                    const uintptr_t src = (uintptr_t)x.p + (uintptr_t)(place(x, t) * (int64_t)sizeof(T)) + (uint64_t)(uint32_t)h * x.head_bytes;
                    const T *head = reinterpret_cast<const T *>(s_ring + at * STEP + (src & 15));
#pragma unroll
                    for (int i = 0; i < UPL; ++i) {
                        if (wanted >> i & 1) xa[i] = *reinterpret_cast<const V *>(head + at_a[i]);
                        if (both >> i & 1) xb[i] = *reinterpret_cast<const V *>(head + at_b[i]);
                    }
                    __syncwarp();  // before the words are copied over
                } else {
#pragma unroll
                    for (int i = 0; i < UPL; ++i) {
                        xa[i] = *reinterpret_cast<const V *>(s_ring + at * STEP + 2 * i * 32 * VB);
                        xb[i] = *reinterpret_cast<const V *>(s_ring + at * STEP + (2 * i + 1) * 32 * VB);
                    }
                }
                at = at + 1 == RING ? 0 : at + 1;
                copy_ahead();
                f(xa, xb, h);
            }
        };
        // Heads turned and stored in the inputs' type, from the element `row` of y on.
        auto move = [&](const Heads &x, const Heads &y, int64_t row, int n, uint32_t wanted, uint32_t both, uint32_t turned,
                        const int (&at_a)[UPL], const int (&at_b)[UPL]) {
            steps(x, n, wanted, both, at_a, at_b, [&](V (&xa)[UPL], V (&xb)[UPL], int h) {
                if (!pos_ok || h >= n || row < 0) return;
                T *dst = reinterpret_cast<T *>((unsigned char *)y.p + (row * (int64_t)sizeof(T) + (uint64_t)(uint32_t)h * y.head_bytes));
#pragma unroll
                for (int i = 0; i < UPL; ++i)
                    if (wanted >> i & 1) {
                        if (turned >> i & 1) {
                            float fa[VE], fb[VE] = {};
                            unpack_raw<T, VB>(xa[i], fa);
                            if (both >> i & 1) unpack_raw<T, VB>(xb[i], fb);
                            turn(i, fa, fb);
                            xa[i] = pack_raw<T, VB>(fa);
                            xb[i] = pack_raw<T, VB>(fb);
                        }
                        *reinterpret_cast<V *>(dst + at_a[i]) = xa[i];
                        if (both >> i & 1) *reinterpret_cast<V *>(dst + at_b[i]) = xb[i];
                    }
            });
        };
        move(a.q, a.q_out, place(a.q_out, t), a.Hq, q_in, two, turns, ia, ib);
        if constexpr (SAME) {
            move(a.k, a.k_out, !a.slots ? place(a.k_out, t) : kept ? slot * a.k_out.st : -1, a.Hkv, k_in, two, turns, ia, ib);
            if (a.slots) move(a.v, a.v_out, kept ? slot * a.v_out.st : -1, a.Hkv, v_in, v_two, 0u, va, vb);
            continue;
        }
        auto quantise = [&](const Heads &x, const Heads &cache, const Scales &scales, uint32_t wanted, uint32_t both, uint32_t turned,
                            const int (&at_a)[UPL], const int (&at_b)[UPL]) {
            steps(x, a.Hkv, wanted, both, at_a, at_b, [&](V (&xa)[UPL], V (&xb)[UPL], int h) {
                if (!pos_ok || !kept) return;
                const bool mine = h < a.Hkv;
                // Several units are turned again behind the maximum: their values in
                // registers would spill.
                constexpr bool HOLD = UPL == 1;
                float fa[VE], fb[VE], top = 0.f;
                auto values = [&](int i) {
                    unpack_raw<T, VB>(xa[i], fa);
#pragma unroll
                    for (int e = 0; e < VE; ++e) fb[e] = 0.f;
                    if (both >> i & 1) unpack_raw<T, VB>(xb[i], fb);
                    if (turned >> i & 1) turn(i, fa, fb);
                };
#pragma unroll
                for (int i = 0; i < UPL; ++i)
                    if (mine && (wanted >> i & 1)) {
                        values(i);
#pragma unroll
                        for (int e = 0; e < VE; ++e) top = max_abs(top, fa[e], fb[e]);
                    }
                const float most = scaled_top<FMT>(head_max(top));
                const float2 by = code_factor<FMT>(most);
                if (!mine || hs >= hpi) return;
                unsigned char *dst = (unsigned char *)cache.p + (slot * cache.st + (uint64_t)(uint32_t)h * cache.head_bytes);
#pragma unroll
                for (int i = 0; i < UPL; ++i)
                    if (wanted >> i & 1) {
                        if constexpr (!HOLD) {
                            same_bits(xa[i]);
                            same_bits(xb[i]);
                            values(i);
                        }
                        *reinterpret_cast<Codes *>(dst + at_a[i]) = code_word<FMT>(fa, by);
                        if (both >> i & 1) *reinterpret_cast<Codes *>(dst + at_b[i]) = code_word<FMT>(fb, by);
                    }
                if (lu == 0) scales.p[slot * scales.st + h * scales.sh] = most * (1.f / top_code<FMT>());
            });
        };
        if constexpr (!SAME) {
            quantise(a.k, a.k_out, a.k_scale, in, two, turns, ia, ib);
            quantise(a.v, a.v_out, a.v_scale, v_in, v_two, 0u, va, vb);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Heads of over 512 elements that are not in 16-byte units (in 4-byte units too; and
// interleaved ones of 1024 with an odd number of vectors in both parts), which have more
// lanes than the ring's instances for smaller units: a warp a head of a token, a lane its
// elements 32 apart, which a head of k or v computes twice, for its largest and for its codes.
// Each head computes its cosines anew: 4096 tokens of 8 + 2 heads of 1022 take 482 us (6 % of
// the copy bandwidth; heads of 512 in 4-byte units 32, of 1024 in 16-byte units 37).
template <typename T, int FMT, bool INTERLEAVED>
__global__ void __launch_bounds__(C8_NT) append8_generic_kernel(const __grid_constant__ AppendArgs a) {
    const int lane = threadIdx.x & 31, half = a.rot / 2;
    const int heads = a.Hq + 2 * a.Hkv;
    const int64_t n_items = a.T * heads, n_warps = (int64_t)gridDim.x * (C8_NT / 32);
    griddep_wait();
    griddep_launch_dependents();
    for (int64_t item = ((int64_t)blockIdx.x * C8_NT + threadIdx.x) >> 5; item < n_items; item += n_warps) {
        const int64_t t = item / heads, slot = a.slots[t];
        const int h = (int)(item - t * heads);
        float2 pos[RX_MAX_AXES];
        bool pos_ok = true;
        for (int x = 0; x < RX_MAX_AXES; ++x) {
            const int64_t p = x < a.axes.n ? a.positions[x * a.T + t] : 0;
            pos[x] = split_position(p);
            pos_ok = pos_ok && p >= 0;
        }
        const bool slot_ok = slot < a.num_slots;
        if ((!pos_ok || !slot_ok) && lane == 0 && h == 0) atomicOr(a.status, BAD_INDEX);
        if (!pos_ok) continue;
        const int what = h < a.Hq ? 0 : h < a.Hq + a.Hkv ? 1 : 2, hk = h - (what == 0 ? 0 : what == 1 ? a.Hq : a.Hq + a.Hkv);
        if (what && (!slot_ok || slot < 0)) continue;
        const Heads &src = what == 0 ? a.q : what == 1 ? a.k : a.v;
        const T *x = static_cast<const T *>(src.p) + t * src.st + hk * src.sh;
        const int rot = what == 2 ? 0 : a.rot;  // v is copied
        // f(i, x_i, j, x_j) for each pair, f(i, x_i, -1, 0) for each element behind them
        auto each = [&](auto f) {
            for (int m = lane; m < rot / 2; m += 32) {
                const int i = INTERLEAVED ? 2 * m : m, j = INTERLEAVED ? i + 1 : m + half;
                float2 p = pos[0];
                for (int n = 1; n < RX_MAX_AXES; ++n) p = a.axes.of[m] == n ? pos[n] : p;
                const float2 cs = cos_sin<true>(p, a.turns[m]);
                const float c = cs.x * a.scale, s = cs.y * a.scale;
                const float u = Cvt<T>::load1(x + i), w = Cvt<T>::load1(x + j);
                f(i, fmaf(-w, s, u * c), j, fmaf(u, s, w * c));
            }
            for (int i = rot + lane; i < a.Dh; i += 32) f(i, Cvt<T>::load1(x + i), -1, 0.f);
        };
        if (what == 0) {
            T *o = static_cast<T *>(const_cast<void *>(a.q_out.p)) + t * a.q_out.st + hk * a.q_out.sh;
            each([&](int i, float u, int j, float w) {
                Cvt<T>::store1(o + i, u);
                if (j >= 0) Cvt<T>::store1(o + j, w);
            });
            continue;
        }
        float top = 0.f;
        each([&](int, float u, int, float w) { top = max_abs(top, u, w); });
        const float most = scaled_top<FMT>(warp_max(top));
        const float2 by = code_factor<FMT>(most);
        const Heads &dst = what == 1 ? a.k_out : a.v_out;
        uint8_t *o = static_cast<uint8_t *>(const_cast<void *>(dst.p)) + slot * dst.st + hk * dst.sh;
        each([&](int i, float u, int j, float w) {
            const uint32_t c = code_pair<FMT>(in_codes(u, by), in_codes(w, by));
            o[i] = (uint8_t)c;
            if (j >= 0) o[j] = (uint8_t)(c >> 8);
        });
        const Scales &sc = what == 1 ? a.k_scale : a.v_scale;
        if (lane == 0) sc.p[slot * sc.st + hk * sc.sh] = most * (1.f / top_code<FMT>());
    }
}

struct ReadArgs {
    Heads k, v, k_out, v_out;  // caches in codes, outputs in elements
    Scales k_scale, v_scale;
    const int64_t *slots;
    int64_t T, num_slots;
    int Hkv, Dh;
    unsigned int *status;
};

// C codes as one load, and C elements as one store.
template <int C> struct CodeLoad;
template <> struct CodeLoad<8> { using type = uint2; };
template <> struct CodeLoad<4> { using type = uint32_t; };
template <> struct CodeLoad<2> { using type = uint16_t; };
template <> struct CodeLoad<1> { using type = uint8_t; };

// Codes are read once; those of less than a sector a warp are met again.
template <int C> __device__ __forceinline__ typename CodeLoad<C>::type load_codes(const typename CodeLoad<C>::type *p) {
    if constexpr (C >= 4) return __ldcs(p);
    else return *p;
}

template <typename T, int FMT, int C>
__device__ __forceinline__ void write_values(T *out, const typename CodeLoad<C>::type &codes, float by) {
    uint32_t w[(C + 3) / 4] = {};
    memcpy(w, &codes, sizeof(codes));
    float f[C < 2 ? 2 : C];
#pragma unroll
    for (int i = 0; i < (C + 1) / 2; ++i) {
        const float2 v = f2mul(value_pair<FMT>(w[i / 2] >> (16 * (i % 2)) & 0xffffu), make_float2(by, by));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
    if constexpr (C == vec_elems<T>()) {
        __stcs(reinterpret_cast<uint4 *>(out), pack_vec<T>(f));  // read once, and far behind in a long context
    } else if constexpr (C == 1) {
        Cvt<T>::store1(out, f[0]);
    } else if constexpr (sizeof(T) == 4) {  // C == 2
        *reinterpret_cast<float2 *>(out) = make_float2(f[0], f[1]);
    } else if constexpr (C == 4) {
        *reinterpret_cast<uint2 *>(out) = make_uint2(Cvt<T>::pack2(f[0], f[1]), Cvt<T>::pack2(f[2], f[3]));
    } else {
        *reinterpret_cast<uint32_t *>(out) = Cvt<T>::pack2(f[0], f[1]);
    }
}

// Rounds of heads (or tokens) of k, and as many of v, that a warp has in flight.  Reading
// further ahead holds up the writes (65536 tokens of 8 heads of 128, bf16: 65 us with two
// rounds, 72 with four), but rounds in small units have few bytes each (16384 tokens of 8
// heads of 90: 31 us with two, 27 with four).
template <int C> __host__ __device__ constexpr int read8_rounds() { return C >= 4 ? 2 : 4; }
constexpr int R8_CTAS_PER_SM = 4, R8_SMALL_CTAS_PER_SM = 3;  // with four rounds of tokens: 80 registers

// A warp takes a token's k and v, or one of a token's `wpt` parts: 32 / cw heads of each a
// round, cw lanes a head and C codes a lane.  A lane's C codes become one store of 16 bytes
// or less, so that a warp's stores fill their lines (with 16 codes and two stores a lane
// 65536 tokens of 8 heads of 128 took 75 us).
template <typename T, int FMT, int C>
__global__ void __launch_bounds__(C8_NT, R8_CTAS_PER_SM) read8_kernel(const __grid_constant__ ReadArgs a, int cw, int wpt) {
    using L = typename CodeLoad<C>::type;
    constexpr int R = read8_rounds<C>();
    const int lane = threadIdx.x & 31, U = a.Dh / C, hpi = 32 / cw, hs = lane / cw, lu = lane - hs * cw;
    const int step = hpi * wpt;  // heads a round
    const int64_t n_items = a.T * wpt, n_warps = (int64_t)gridDim.x * (C8_NT / 32);
    const int shift = 31 - __clz(wpt);  // wpt is a power of two
    griddep_wait();
    griddep_launch_dependents();
    int64_t w = ((int64_t)blockIdx.x * C8_NT + threadIdx.x) >> 5, next = w < n_items ? a.slots[w >> shift] : 0;
    for (; w < n_items; w += n_warps) {
        const int64_t t = w >> shift, slot = next;
        const int part = (int)(w & (wpt - 1));
        if (w + n_warps < n_items) next = a.slots[(w + n_warps) >> shift];
        const bool there = slot >= 0 && slot < a.num_slots;
        if (slot >= a.num_slots && lane == 0 && part == 0) atomicOr(a.status, BAD_INDEX);
        if (hs >= hpi) continue;
        const int h0 = part * hpi + hs;
        const uint8_t *k = static_cast<const uint8_t *>(a.k.p) + (slot * a.k.st + h0 * a.k.sh);
        const uint8_t *v = static_cast<const uint8_t *>(a.v.p) + (slot * a.v.st + h0 * a.v.sh);
        const float *ks = a.k_scale.p + (slot * a.k_scale.st + h0 * a.k_scale.sh);
        const float *vs = a.v_scale.p + (slot * a.v_scale.st + h0 * a.v_scale.sh);
        T *ko = static_cast<T *>(const_cast<void *>(a.k_out.p)) + (t * a.k_out.st + h0 * a.k_out.sh);
        T *vo = static_cast<T *>(const_cast<void *>(a.v_out.p)) + (t * a.v_out.st + h0 * a.v_out.sh);
        for (int h = h0; h < a.Hkv; h += R * step) {
            float kb[R], vb[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const bool in = there && h + i * step < a.Hkv;
                kb[i] = in ? ks[i * step * a.k_scale.sh] : 0.f;
                vb[i] = in ? vs[i * step * a.v_scale.sh] : 0.f;
            }
            for (int u = lu; u < U; u += cw) {
                L kc[R], vc[R];
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    kc[i] = L{};
                    vc[i] = L{};
                    if (there && h + i * step < a.Hkv) {
                        kc[i] = load_codes<C>(reinterpret_cast<const L *>(k + i * step * a.k.sh + u * C));
                        vc[i] = load_codes<C>(reinterpret_cast<const L *>(v + i * step * a.v.sh + u * C));
                    }
                }
#pragma unroll
                for (int i = 0; i < R; ++i)
                    if (h + i * step < a.Hkv) {
                        write_values<T, FMT, C>(ko + i * step * a.k_out.sh + u * C, kc[i], kb[i]);
                        write_values<T, FMT, C>(vo + i * step * a.v_out.sh + u * C, vc[i], vb[i]);
                    }
            }
            k += R * step * a.k.sh;
            v += R * step * a.v.sh;
            ks += R * step * a.k_scale.sh;
            vs += R * step * a.v_scale.sh;
            ko += R * step * a.k_out.sh;
            vo += R * step * a.v_out.sh;
        }
    }
}

// Tokens of few heads: a round is all heads of `tokens` tokens, and the rounds are dealt
// out to the warps in turn (60000 tokens of 2 heads of 64: 24 us with a warp a token, 11 so).
template <typename T, int FMT, int C>
__global__ void __launch_bounds__(C8_NT, R8_SMALL_CTAS_PER_SM) read8_tokens_kernel(const __grid_constant__ ReadArgs a, int cw, int tokens) {
    using L = typename CodeLoad<C>::type;
    constexpr int R = read8_rounds<C>();
    const int lane = threadIdx.x & 31, U = a.Dh / C, hs = lane / cw, lu = lane - hs * cw;
    const int sub = hs / a.Hkv, h = hs - sub * a.Hkv;  // this lane's token within a round, and head
    const bool in = sub < tokens;
    const int64_t step = (int64_t)gridDim.x * (C8_NT / 32) * tokens;  // tokens of all warps' rounds
    int64_t t = (((int64_t)blockIdx.x * C8_NT + threadIdx.x) >> 5) * tokens + sub, slot[R];
    griddep_wait();
    griddep_launch_dependents();
#pragma unroll
    for (int i = 0; i < R; ++i) slot[i] = in && t + i * step < a.T ? a.slots[t + i * step] : -1;
    for (; t - sub < a.T; t += R * step) {  // the same in a warp's lanes
        int64_t at[R];
        float kb[R], vb[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            at[i] = slot[i];
            const int64_t next = t + (R + i) * step;  // its slot a trip to memory early
            slot[i] = in && next < a.T ? a.slots[next] : -1;
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (at[i] >= a.num_slots) {
                if (lu == 0) atomicOr(a.status, BAD_INDEX);
                at[i] = -1;
            }
            kb[i] = at[i] >= 0 ? a.k_scale.p[at[i] * a.k_scale.st + h * a.k_scale.sh] : 0.f;
            vb[i] = at[i] >= 0 ? a.v_scale.p[at[i] * a.v_scale.st + h * a.v_scale.sh] : 0.f;
        }
        for (int u = lu; u < U; u += cw) {
            L kc[R], vc[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                kc[i] = L{};
                vc[i] = L{};
                if (at[i] >= 0) {
                    kc[i] = load_codes<C>(reinterpret_cast<const L *>(static_cast<const uint8_t *>(a.k.p) + (at[i] * a.k.st + h * a.k.sh)) + u);
                    vc[i] = load_codes<C>(reinterpret_cast<const L *>(static_cast<const uint8_t *>(a.v.p) + (at[i] * a.v.st + h * a.v.sh)) + u);
                }
            }
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (in && t + i * step < a.T) {
                    const int64_t to = t + i * step;
                    write_values<T, FMT, C>(static_cast<T *>(const_cast<void *>(a.k_out.p)) + (to * a.k_out.st + h * a.k_out.sh + u * C), kc[i], kb[i]);
                    write_values<T, FMT, C>(static_cast<T *>(const_cast<void *>(a.v_out.p)) + (to * a.v_out.st + h * a.v_out.sh + u * C), vc[i], vb[i]);
                }
        }
    }
}

}  // namespace rmsn
