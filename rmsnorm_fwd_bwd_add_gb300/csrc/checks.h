// checks.h -- argument checks shared by the entry points: scalars and shapes, row
// strides, alignment, and the overlap rules between row tensors and buffers.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "rmsnorm.h"

namespace rmsn {

inline int esize_of(int dtype) { return dtype == RMSNORM_F32 ? 4 : 2; }

// Scalar and shape checks common to every norm entry point.
inline int check_common(int64_t rows, int64_t D, int dtype, float eps, float weight_bias) {
    if (dtype != RMSNORM_F16 && dtype != RMSNORM_BF16 && dtype != RMSNORM_F32)
        return RMSNORM_ERR_INVALID_ARG;
    if (rows < 0 || D <= 0) return RMSNORM_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return RMSNORM_ERR_INVALID_ARG;
    if (!std::isfinite(weight_bias)) return RMSNORM_ERR_INVALID_ARG;
    if (D > RMSNORM_MAX_D) return RMSNORM_ERR_UNSUPPORTED;
    if (rows > INT64_MAX / (4 * D)) return RMSNORM_ERR_UNSUPPORTED;
    return RMSNORM_OK;
}

inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t pa = (uintptr_t)a, pb = (uintptr_t)b;
    return pa < pb + nb && pb < pa + na;
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// A [rows, D] tensor of `es`-byte elements whose rows start `ld` elements
// apart (ld >= D).  A single row has no stride; it is normalised to D so
// that the same row under two strides compares equal.
struct Mat {
    const void *p;
    int64_t ld;
};

inline Mat mat(const void *p, int64_t ld, int64_t rows, int64_t D) { return Mat{p, rows <= 1 ? D : ld}; }

// Checks a stride and that the tensor's extent fits in the address space.
inline int check_ld(int64_t ld, int64_t rows, int64_t D, int es) {
    if (ld < D) return RMSNORM_ERR_INVALID_ARG;
    if (rows > 1 && (rows - 1) > (INT64_MAX / es - D) / ld) return RMSNORM_ERR_UNSUPPORTED;
    return RMSNORM_OK;
}

inline size_t extent(const Mat &m, int64_t rows, int64_t D, int es) {
    return (!m.p || rows == 0) ? 0 : (size_t)((rows - 1) * m.ld + D) * (size_t)es;
}

inline int64_t floor_div(int64_t a, int64_t b) {
    const int64_t q = a / b;
    return (a % b != 0 && ((a < 0) != (b < 0))) ? q - 1 : q;
}

// Whether two [rows, D] tensors share a byte.  With equal strides the test is
// exact (rows i of a and j of b meet iff |(b - a) - (i - j) * ld| < the row's
// bytes for some i - j in [-(rows - 1), rows - 1]), so interleaved tensors
// such as the two halves of a [rows, 2D] buffer count as disjoint; with
// different strides the whole extents are compared.
inline bool mats_overlap(const Mat &a, const Mat &b, int64_t rows, int64_t D, int es) {
    const size_t na = extent(a, rows, D, es), nb = extent(b, rows, D, es);
    if (!overlaps(a.p, na, b.p, nb)) return false;
    if (a.ld != b.ld) return true;
    const int64_t L = a.ld * es, R = D * es;
    const int64_t d = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p);
    const int64_t k0 = floor_div(d, L);
    for (int64_t k : {k0, k0 + 1}) {
        k = std::min<int64_t>(std::max<int64_t>(k, -(rows - 1)), rows - 1);
        const int64_t off = d - k * L;
        if (off > -R && off < R) return true;
    }
    return false;
}

// An output may be exactly an input (same pointer and stride: every element
// is read before the thread that owns it writes it), or share no byte with it.
inline bool bad_alias(const Mat &out, const Mat &in, int64_t rows, int64_t D, int es) {
    if (!mats_overlap(out, in, rows, D, es)) return false;
    return !(out.p == in.p && out.ld == in.ld);
}

// Whether a [rows, D] tensor overlaps a plain buffer of n bytes.
inline bool mat_hits(const Mat &m, int64_t rows, int64_t D, int es, const void *p, size_t n) {
    return overlaps(m.p, extent(m, rows, D, es), p, n);
}

// The vectorised tiers need 16-byte aligned rows: base and stride.
inline bool rows_aligned(const Mat &m, int es) {
    return !m.p || (aligned16(m.p) && (m.ld * es) % 16 == 0);
}

// Every element of every operand must sit at a multiple of its size.
inline bool elem_aligned(const void *p, int es) { return ((uintptr_t)p % (uintptr_t)es) == 0; }

}  // namespace rmsn
