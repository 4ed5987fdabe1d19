// selective_scan.cuh -- internal interface of the selective scan, and what its kernels share.
//
// For sequence b, channel d (of group g = d / (D / G)) and state n, with s_t = softplus(dt_t + dt_bias) or dt_t + dt_bias:
//
//   h_t = exp(s_t a) h_(t-1) + s_t x_t b_t[g, n],   y_t = (sum_n c_t[g, n] h_t[n] + skip x_t) silu(gate_t)
//
// and backward, with v_t = dy_t silu(gate_t) and P the gradient that arrives at the state before a token:
//
//   G_t = P_(t+1) + v_t c_t,   P_t = exp(s_t a) G_t,   P_(T+1) = dh
//   dc_t = sum_d v_t h_t,      db_t = sum_d G_t s_t x_t,   dx_t = s_t sum_n G_t b_t + skip v_t
//   ds_t = sum_n a P_t h_(t-1) + x_t sum_n G_t b_t,        da = sum_(b, t) s_t P_t h_(t-1),    dh0 = P_1
//
// Both are affine recurrences; where there are few of them, time is split into segments: a first pass leaves each
// segment's own last state and the sum of its s (the segment's decay is exp(a sum s)), a join makes the states that the
// segments start from, and the last pass runs all segments at once.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "solver.cuh"

namespace pararnn {

constexpr int kSsKeep = 8;  // tokens between the states that the forward pass keeps for the backward pass

struct SsRows {  // [B, T, D] or [B, T, G, N] operand: element strides, innermost contiguous; p may be null
    const void *p;
    long long sb, st, sg;
};

struct SsArgs {
    int B, T, D, G, N, dtype, softplus;
    SsRows x, dt, b, c, gate, dy;
    const float *a, *skip, *dt_bias, *h0, *dh;
    const int *lengths;
    void *y;
    float *h;     // [B, D, N]
    float *kept;  // [B, ceil(T / 8), D, N]: the state before every 8th token, or null
    int n_seg, seg;            // segments of `seg` tokens (a multiple of 16)
    float *seg_state, *seg_dt;  // [n_seg, B, D, N], [n_seg, B, D]
    // backward
    float *rev_state;  // [n_seg, B, D, N]: P behind each segment
    void *dx, *ddt, *dgate, *db, *dc;
    float *da, *dskip, *ddt_bias, *dh0;
    float *part_b, *part_c;                // [tiles of a group, B, T, G, N]
    float *part_a, *part_skip, *part_bias;  // [n_seg, B, D, N], [n_seg, B, D]
};

struct SsPlan {
    int n_seg, seg;
};
SsPlan ss_plan(const SsArgs &a, bool backward);
int ss_backward_tiles(const SsArgs &a);  // CTAs along a group's channels in the backward pass
cudaError_t launch_ss_forward(const SsArgs &a, cudaStream_t s);
cudaError_t launch_ss_kept(const SsArgs &a, cudaStream_t s);  // the kept states alone
cudaError_t launch_ss_reverse_states(const SsArgs &a, cudaStream_t s);  // rev_state, where there are segments
cudaError_t launch_ss_backward(const SsArgs &a, cudaStream_t s);

struct SsStep {
    int B, D, G, N, dtype, softplus, n_slots;
    SsRows x, dt, b, c, gate;  // st unused
    const float *a, *skip, *dt_bias, *state;
    const int *slots;
    void *y;
    float *out_state;
};
cudaError_t launch_ss_step(const SsStep &w, cudaStream_t s);

// ---- device helpers -----------------------------------------------------------------------------------------

namespace ss {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16(x); }

__device__ __forceinline__ int row_count(const int *lengths, int b, int T) {
    if (lengths == nullptr) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : (n > T ? T : n);
}

__device__ __forceinline__ float softplus(float v) { return v > 20.f ? v : log1pf(expf(v)); }
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + expf(-v)); }
__device__ __forceinline__ float gate_with(float y, float z) { return y * (z * sigmoid(z)); }

// exp(s a) - 1 for a pair of states, from x = s a log2(e).  The state is updated as h + (exp(s a) - 1) h: rounded to fp32,
// exp(s a) of a slow decay would be another decay, taken at every token.  Near zero the difference comes from its series
// (the first term left out is below (ln 2 / 16)^4 / 120 = 3e-8 of it), further away from ex2, whose 1.3e-7 is then below
// 3e-6 of it.
__device__ __forceinline__ u64 decay_less_one(u64 x) {
    const u64 p = mul2(x, fma2(x, fma2(x, fma2(x, splat(0.00961812910f), splat(0.0555041087f)), splat(0.240226507f)),
                               splat(0.693147181f)));
    const u64 e = add2(ex2_2(x), splat(-1.f));
    float x0, x1, p0, p1, e0, e1;
    upk(x, x0, x1), upk(p, p0, p1), upk(e, e0, e1);
    return pk(fabsf(x0) < 0.0625f ? p0 : e0, fabsf(x1) < 0.0625f ? p1 : e1);
}

template <int PAIRS>
__device__ __forceinline__ void load_pairs(u64 (&v)[PAIRS], const float *p) {
    if constexpr (PAIRS % 2 == 0) {
#pragma unroll
        for (int i = 0; i < PAIRS; i += 2) {
            const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(p + 2 * i);
            v[i] = q.x, v[i + 1] = q.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) v[i] = *reinterpret_cast<const u64 *>(p + 2 * i);
    }
}
// states n0 .. of [.., N] fp32 rows in global memory; zero behind N
template <int PAIRS>
__device__ __forceinline__ void load_states(u64 (&v)[PAIRS], const float *p, int n0, int N, bool vec) {
    if (vec) {
#pragma unroll
        for (int i = 0; i < PAIRS; i += 2) {
            const float4 q = n0 + 2 * i < N ? *reinterpret_cast<const float4 *>(p + n0 + 2 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[i] = pk(q.x, q.y), v[i + 1] = pk(q.z, q.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const int n = n0 + 2 * i;
            v[i] = pk(n < N ? p[n] : 0.f, n + 1 < N ? p[n + 1] : 0.f);
        }
    }
}
template <int PAIRS>
__device__ __forceinline__ void store_states(const u64 (&v)[PAIRS], float *p, int n0, int N, bool vec) {
#pragma unroll
    for (int i = 0; i < PAIRS; i += 2) {
        float q[4];
        upk(v[i], q[0], q[1]), upk(v[i + 1], q[2], q[3]);
        const int n = n0 + 2 * i;
        if (vec) {
            if (n < N) *reinterpret_cast<float4 *>(p + n) = make_float4(q[0], q[1], q[2], q[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < N) p[n + j] = q[j];
        }
    }
}
__device__ __forceinline__ float pair_sum(u64 v) {
    float a, b;
    upk(v, a, b);
    return a + b;
}

}  // namespace ss
}  // namespace pararnn
