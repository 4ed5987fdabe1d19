// layer_norm.cuh -- internal interface of the residual stream's norm: add a branch, store the sum, normalise its rows.
#pragma once

#include "solver.cuh"

namespace pararnn {

struct LnArgs {
    int N, S, C, x_dtype, r_dtype, y_dtype, rms;
    float eps;
    const void *x, *residual;    // forward: x of x_dtype, residual of r_dtype or null
    const float *weight, *bias;  // [C] or null
    const int *lengths;          // [N] or null
    void *y, *r;                 // forward: r null without a residual; backward: y is dy, r the stream (both read)
    float *stats;                // [N, S, 2]
    // backward
    const void *dr_in;  // of r_dtype, or null
    void *dr, *dx;      // of r_dtype; of x_dtype, or null
    float *dweight, *dbias;
    float *part;  // [ln_backward_rows, 2 C]
};
int ln_backward_rows(const LnArgs &a);
cudaError_t launch_ln_forward(const LnArgs &a, cudaStream_t s);
cudaError_t launch_ln_backward(const LnArgs &a, cudaStream_t s);

}  // namespace pararnn
