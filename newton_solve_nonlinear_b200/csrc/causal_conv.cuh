// causal_conv.cuh -- internal interface of the short causal convolution over time, one filter per channel.
#pragma once

#include "solver.cuh"

namespace pararnn {

struct CcRows {  // [B, T, D]: element strides, innermost contiguous
    const void *p;
    long long sb, st;
};

struct CcArgs {
    int B, T, D, W, dtype, act;
    CcRows x, dy;
    const float *weight, *bias;  // [D, W]; [D] or null
    const void *state, *dlast;   // [B, W - 1, D] or null
    const int *lengths;
    void *y, *last;
    // backward
    void *dx, *dstate;
    float *dweight, *dbias;
    float *part;  // [cc_backward_rows, D, W + 1]
};
int cc_backward_rows(const CcArgs &a);
cudaError_t launch_cc_forward(const CcArgs &a, cudaStream_t s);
cudaError_t launch_cc_backward(const CcArgs &a, cudaStream_t s);

struct CcStep {
    int B, D, W, dtype, act, n_slots;
    CcRows x;  // st unused
    const float *weight, *bias;
    const void *state;
    const int *slots;
    void *y, *out_state;
};
cudaError_t launch_cc_step(const CcStep &w, cudaStream_t s);

}  // namespace pararnn
