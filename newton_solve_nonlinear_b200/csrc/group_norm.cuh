// group_norm.cuh -- internal interface of group norm with an activation or a gate, channels last.
#pragma once

#include "solver.cuh"

namespace pararnn {

struct GnArgs {
    int N, S, C, G;
    int x_dtype, y_dtype, act;
    float eps;
    const void *x, *gate;        // [N, S, C] of x_dtype; gate may be null
    const float *weight, *bias;  // [C] or null
    const int *lengths;          // [N] or null
    float *stats;                // [N, G, 2]: mean and 1 / sqrt(var + eps)
    void *y;                     // forward: out; backward: dy (read), of y_dtype
    void *dx, *dgate;            // backward
    float *dweight, *dbias;
    char *ws;
};

size_t gn_ws_bytes(const GnArgs &a, bool backward);
cudaError_t launch_gn_forward(const GnArgs &a, cudaStream_t s);
cudaError_t launch_gn_backward(const GnArgs &a, cudaStream_t s);

}  // namespace pararnn
