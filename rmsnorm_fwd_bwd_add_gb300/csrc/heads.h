// heads.h -- operands of the rotary and cache calls, [B, S, H, Dh] with a stride for
// each of the outer dimensions: their extents, alignment and overlaps (host; the
// struct is the kernels' too).
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "checks.h"

namespace rmsn {

// One tensor [B, S, H, Dh]: strides in elements, Dh contiguous; and the head stride
// in bytes, below 2^32, so that a head's address is one multiply-add.
struct Heads {
    const void *p;
    int64_t sb, st, sh;
    uint32_t head_bytes;
};

// A [B, S, H, Dh] operand: whether its strides are usable, the bytes it spans,
// and for outputs that no two of its elements share an address.
struct Span {
    uintptr_t lo, hi;   // bytes [lo, hi)
    Mat m;              // as rows of one token (or one batch) each, a stride apart
    int64_t row;        // elements from such a row's first to its last, 0 if there is no such stride
};

inline bool safe_mul_add(int64_t n, int64_t st, int64_t *sum) {  // *sum += (n - 1) * st
    if (n > 1 && st > ((int64_t)1 << 60) / (n - 1)) return false;
    *sum += n > 1 ? (n - 1) * st : 0;
    return *sum < ((int64_t)1 << 60);
}

inline int span_of(const Heads &h, int64_t B, int64_t S, int64_t H, int64_t Dh, int es, bool output, Span *out) {
    *out = Span{0, 0, Mat{nullptr, 0}, 0};
    if (!h.p || B * S == 0 || H == 0) return RMSNORM_OK;
    if (!elem_aligned(h.p, es) || h.sb < 0 || h.st < 0 || h.sh < 0) return RMSNORM_ERR_INVALID_ARG;
    if (H > 1 && h.sh > (int64_t)UINT32_MAX / es) return RMSNORM_ERR_UNSUPPORTED;
    int64_t last = Dh - 1;
    if (!safe_mul_add(B, h.sb, &last) || !safe_mul_add(S, h.st, &last) || !safe_mul_add(H, h.sh, &last))
        return RMSNORM_ERR_UNSUPPORTED;
    if (output) {  // in order of stride, each dimension steps past the ones inside it
        struct { int64_t n, st; } d[3] = {{B, h.sb}, {S, h.st}, {H, h.sh}};
        std::sort(d, d + 3, [](auto &x, auto &y) { return x.st < y.st; });
        int64_t inner = Dh;
        for (auto &x : d) {
            if (x.n <= 1) continue;
            if (x.st < inner) return RMSNORM_ERR_INVALID_ARG;
            inner += (x.n - 1) * x.st;
        }
    }
    out->lo = (uintptr_t)h.p;
    out->hi = out->lo + (size_t)(last + 1) * es;
    const int64_t foot = (H - 1) * h.sh + Dh;
    const int64_t st = S > 1 ? h.st : h.sb;  // one stride from token to token
    if ((B == 1 || S == 1 || h.sb == S * h.st) && (B * S == 1 || st >= foot)) {
        out->m = mat(h.p, st, B * S, foot);
        out->row = foot;
    } else if (B > 1) {  // heads outside tokens: one stride from batch to batch
        const int64_t whole = (H - 1) * h.sh + (S - 1) * h.st + Dh;
        if (h.sb >= whole) {
            out->m = Mat{h.p, h.sb};
            out->row = whole;
        }
    }
    return RMSNORM_OK;
}

// Whether two operands, with elements of ea and eb bytes, may share a byte: by their
// rows where these are a common stride apart (heads of one fused projection, codes
// and scales of one slot), by whole spans otherwise.
inline bool spans_meet(const Span &a, int ea, const Span &b, int eb) {
    if (a.hi <= b.lo || b.hi <= a.lo) return false;
    if (!a.row || !b.row || a.m.ld * ea != b.m.ld * eb) return true;
    const int64_t L = a.m.ld * ea;
    int64_t r = (int64_t)(b.lo - a.lo) % L;
    if (r < 0) r += L;  // b's rows start r bytes into a's periods
    return r < a.row * ea || r + b.row * eb > L;
}
inline bool spans_meet(const Span &a, const Span &b, int es) { return spans_meet(a, es, b, es); }

inline bool same_place(const Heads &a, const Heads &b, int64_t B, int64_t S, int64_t H) {
    return a.p == b.p && (B <= 1 || a.sb == b.sb) && (S <= 1 || a.st == b.st) && (H <= 1 || a.sh == b.sh);
}

// The bits of every address and stride in bytes.
inline uintptr_t byte_bits(const Heads &h, int64_t B, int64_t S, int64_t H, int es) {
    if (!h.p) return 0;
    return (uintptr_t)h.p | (uintptr_t)((B > 1 ? h.sb : 0) * es) | (uintptr_t)((S > 1 ? h.st : 0) * es) |
           (uintptr_t)((H > 1 ? h.sh : 0) * es);
}

// The stride of a single head counts for nothing, here as in byte_bits: lanes of a warp
// whose places lie behind the heads form addresses with it, in units that it need not
// divide, and read shared memory there.
inline Heads heads(const void *p, const int64_t *st, int n, int es, int64_t H) {
    // n = 3: batch, token, head; n = 2: token, head
    if (!p || !st) return Heads{nullptr, 0, 0, 0, 0};
    const int64_t sh = H > 1 ? st[n - 1] : 0;
    return Heads{p, n == 3 ? st[0] : 0, st[n - 2], sh, (uint32_t)(sh * es)};
}

}  // namespace rmsn
