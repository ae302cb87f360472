// norm_q8.h -- arguments of the 8-bit norm's kernels.
#pragma once

#include <cstdint>

namespace rmsn {

struct Q8Args {
    const void *x, *res, *w;  // res null: none
    void *out, *nres;         // codes, one byte each; new residual
    float *scale;
    int64_t ld_x, ld_res, ld_out, ld_nres;
    int64_t rows;
    int D, group, groups;  // group: columns of a scale, 0: the row; groups a row
    float eps, weight_bias;
};

}  // namespace rmsn
