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
    float *part_a;                         // [n_seg, B, D N + D + D]: da, dskip and ddt_bias of each segment
};

struct SsPlan {
    int n_seg, seg;
};
SsPlan ss_plan(const SsArgs &a);
bool ss_pairs_ok(const SsArgs &a);       // pairs of channels and quads of b and c on their own alignment
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

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN where either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// A rate as the kernels take it, in powers of two.  -inf is the lowest finite one: it forgets at every token, but where a step
// is zero (in the places behind a sequence, too) nothing decays, and zero times infinity would be NaN.
__device__ __forceinline__ float above_inf(float v) { return max_nan(v, -3.402823466e38f); }
__device__ __forceinline__ float rate_of(float a) { return above_inf(a * kLog2eF); }
// exp(v), |v| at most 150: ex2 of v log2(e) rounded, times what that rounding and log2(e)'s own left out.  (One value at a
// time: a constant of a packed operation takes two registers and two instructions to fill them.)
__device__ __forceinline__ float exp_of(float v) {
    const float t = v * kLog2eF, rest = fmaf(v, 1.92596299e-8f, fmaf(v, kLog2eF, -t));
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    return fmaf(e, rest * 0.693147181f, e);
}
// log(1 + exp(v)) = max(v, 0) + log(1 + e), e = exp(-|v|) in (0, 1]; log(1 + e) / e is a polynomial fitted for the smallest
// largest relative error on [0, 1], 1.6e-7 as evaluated.  -inf gives 0, as the limit does.
// With its slope 1 / (1 + exp(-v)).
__device__ __forceinline__ float softplus(float v, float &slope) {
    const float e = exp_of(max_nan(-fabsf(v), -150.f));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    slope = v >= 0.f ? r : e * r;
    float p = fmaf(0.00523268804f, e, -0.0295052137f);
    p = fmaf(p, e, 0.0782259107f);
    p = fmaf(p, e, -0.136632428f);
    p = fmaf(p, e, 0.191060051f);
    p = fmaf(p, e, -0.24842982f);
    p = fmaf(p, e, 0.333190978f);
    p = fmaf(p, e, -0.499994934f);
    p = fmaf(p, e, 0.99999994f);
    return fmaf(p, e, max_nan(v, 0.f));
}
__device__ __forceinline__ float softplus(float v) {
    float unused;
    return softplus(v, unused);
}
// 1 / (1 + exp(-z)); below -88 it is zero, as exp(88.7) is still finite and its inverse no longer a normal number
__device__ __forceinline__ float sigmoid_of(float z) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + exp_of(min_nan(max_nan(-z, -88.7f), 88.7f))));
    return r;
}
__device__ __forceinline__ float gate_with(float y, float z) { return y * (z * sigmoid_of(z)); }

// Two neighbouring channels' elements, as they lie in memory: fetched long before they are used.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
    unsigned v;
};
template <>
struct Raw<float> {
    u64 v;
};
// VEC: both exist and are aligned as a pair; n of them exist
template <bool VEC>
__device__ __forceinline__ Raw<__nv_bfloat16> load_raw(const __nv_bfloat16 *p, int n) {
    if constexpr (VEC) return {n > 0 ? *reinterpret_cast<const unsigned *>(p) : 0u};
    const unsigned short *q = reinterpret_cast<const unsigned short *>(p);
    return {(n > 0 ? q[0] : 0u) | (n > 1 ? static_cast<unsigned>(q[1]) << 16 : 0u)};
}
template <bool VEC>
__device__ __forceinline__ Raw<float> load_raw(const float *p, int n) {
    if constexpr (VEC) return {n > 0 ? *reinterpret_cast<const u64 *>(p) : 0ull};
    return {pk(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f)};
}
// the same of one or four elements of b or c
template <typename T, int W>
struct RawN;
template <>
struct RawN<__nv_bfloat16, 1> {
    unsigned short v;
};
template <>
struct RawN<__nv_bfloat16, 4> {
    uint2 v;
};
template <>
struct RawN<float, 1> {
    float v;
};
template <>
struct RawN<float, 4> {
    float4 v;
};
template <int W, typename T>
__device__ __forceinline__ RawN<T, W> load_n(const T *p, bool on) {
    RawN<T, W> r{};
    if (on) r = *reinterpret_cast<const RawN<T, W> *>(p);
    return r;
}
__device__ __forceinline__ void store_n(float *p, RawN<__nv_bfloat16, 1> r) {
    *p = __uint_as_float(static_cast<unsigned>(r.v) << 16);
}
__device__ __forceinline__ void store_n(float *p, RawN<__nv_bfloat16, 4> r) {
    *reinterpret_cast<float4 *>(p) = make_float4(__uint_as_float(r.v.x << 16), __uint_as_float(r.v.x & 0xffff0000u),
                                                 __uint_as_float(r.v.y << 16), __uint_as_float(r.v.y & 0xffff0000u));
}
__device__ __forceinline__ void store_n(float *p, RawN<float, 1> r) { *p = r.v; }
__device__ __forceinline__ void store_n(float *p, RawN<float, 4> r) { *reinterpret_cast<float4 *>(p) = r.v; }
__device__ __forceinline__ void unpack_n(float *f, RawN<__nv_bfloat16, 1> r) { *f = __uint_as_float(static_cast<unsigned>(r.v) << 16); }
__device__ __forceinline__ void unpack_n(float *f, RawN<__nv_bfloat16, 4> r) {
    f[0] = __uint_as_float(r.v.x << 16), f[1] = __uint_as_float(r.v.x & 0xffff0000u);
    f[2] = __uint_as_float(r.v.y << 16), f[3] = __uint_as_float(r.v.y & 0xffff0000u);
}
__device__ __forceinline__ void unpack_n(float *f, RawN<float, 1> r) { *f = r.v; }
__device__ __forceinline__ void unpack_n(float *f, RawN<float, 4> r) { f[0] = r.v.x, f[1] = r.v.y, f[2] = r.v.z, f[3] = r.v.w; }
template <int N>
__device__ __forceinline__ void load_floats(float (&v)[N], const float *p) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(p + i);
            v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 q = *reinterpret_cast<const float2 *>(p + i);
            v[i] = q.x, v[i + 1] = q.y;
        }
    }
}
__device__ __forceinline__ u64 value(Raw<__nv_bfloat16> r) {
    return pk(__uint_as_float(r.v << 16), __uint_as_float(r.v & 0xffff0000u));
}
__device__ __forceinline__ u64 value(Raw<float> r) { return r.v; }
template <bool VEC>
__device__ __forceinline__ void store_pair(__nv_bfloat16 *p, u64 v, int n) {
    float a, b;
    upk(v, a, b);
    const __nv_bfloat162 q = __floats2bfloat162_rn(a, b);
    if constexpr (VEC) {
        if (n > 0) *reinterpret_cast<__nv_bfloat162 *>(p) = q;
    } else {
        if (n > 0) p[0] = q.x;
        if (n > 1) p[1] = q.y;
    }
}
template <bool VEC>
__device__ __forceinline__ void store_pair(float *p, u64 v, int n) {
    if constexpr (VEC) {
        if (n > 0) *reinterpret_cast<u64 *>(p) = v;
    } else {
        float a, b;
        upk(v, a, b);
        if (n > 0) p[0] = a;
        if (n > 1) p[1] = b;
    }
}

// A decay takes v to f v + (slow ? v : 0), for a pair of states with x = s a log2(e): f is exp(s a) - 1 where the decay is slow
// and exp(s a) elsewhere.  Rounded to fp32, exp(s a) of a slow decay would be another decay, taken at every token; the
// difference from 1 of a fast one would leave 2^-24 of the old value behind, where exp(s a) may be far below that.  Near zero
// the difference comes from its series (the first term left out is (ln 2 / 64)^3 / 24 = 5e-8 of it), further away exp(s a)
// from ex2, whose 1.3e-7 counts for no more than the 92 tokens that such a state remembers.
__device__ __forceinline__ bool slow_decay(float x) { return fabsf(x) < 0.015625f; }
__device__ __forceinline__ u64 decay_factor(u64 x) {
    const u64 p = mul2(x, fma2(x, fma2(x, splat(0.0555041087f), splat(0.240226507f)), splat(0.693147181f)));
    const u64 e = ex2_2(x);
    float x0, x1, p0, p1, e0, e1;
    upk(x, x0, x1), upk(p, p0, p1), upk(e, e0, e1);
    return pk(slow_decay(x0) ? p0 : e0, slow_decay(x1) ? p1 : e1);
}
// a and b, and what stays beside f v.  (Additions under a condition: selecting what to add takes 3 % of the forward pass.)
__device__ __forceinline__ u64 with_rest(u64 x, float a, float b, u64 v) {
    float x0, x1, v0, v1;
    upk(x, x0, x1), upk(v, v0, v1);
    if (slow_decay(x0)) a += v0;
    if (slow_decay(x1)) b += v1;
    return pk(a, b);
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
template <int PAIRS>
__device__ __forceinline__ void store_pairs(float *p, const u64 (&v)[PAIRS]) {
    if constexpr (PAIRS == 2) *reinterpret_cast<ulonglong2 *>(p) = make_ulonglong2(v[0], v[1]);
    else *reinterpret_cast<u64 *>(p) = v[0];
}
// states n0 .. of [.., N] fp32 rows in global memory; zero behind N.  vec: the row's start and N are multiples of 2 PAIRS
template <int PAIRS>
__device__ __forceinline__ void load_states(u64 (&v)[PAIRS], const float *p, int n0, int N, bool vec) {
    if (vec) {
        if constexpr (PAIRS == 2) {
            const ulonglong2 q = n0 < N ? *reinterpret_cast<const ulonglong2 *>(p + n0) : make_ulonglong2(0, 0);
            v[0] = q.x, v[1] = q.y;
        } else {
            v[0] = n0 < N ? *reinterpret_cast<const u64 *>(p + n0) : 0ull;
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
    if (vec) {
        if (n0 >= N) return;
        if constexpr (PAIRS == 2) *reinterpret_cast<ulonglong2 *>(p + n0) = make_ulonglong2(v[0], v[1]);
        else *reinterpret_cast<u64 *>(p + n0) = v[0];
    } else {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            float a, b;
            upk(v[i], a, b);
            const int n = n0 + 2 * i;
            if (n < N) p[n] = a;
            if (n + 1 < N) p[n + 1] = b;
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
