// linear_attention.cuh -- the sweep that linear attention and its backward pass are made of.
//
// One head of one sequence carries a dk x dv matrix state S.  With g = exp(log_decay[h]) a sweep computes,
// over the logical rows r = 0 .. L-1 (row r is token r, or token L-1-r when `reverse` is set),
//
//   out_r = intra * sum_{s <= r} g^(r-s) (a_r . b_s) c_s  +  inter * g^(r+e) (a_r^T S_in)
//   S_out = g^L S_in + update * sum_s g^(L-e-s) b_s c_s^T
//
//   forward   o  = sweep(a=q,  b=k,  c=v),  e = 1,  S_in = S_0,   intra = inter = scale, update = 1
//   backward  dq = sweep(a=do, b=v,  c=k),  e = 1,  S_in = S_0^T, intra = inter = scale, update = 1
//             dv = sweep(a=k,  b=q,  c=do), reverse, e = 0, S_in = dS,   intra = update = scale, inter = 1
//             dk = sweep(a=v,  b=do, c=q),  reverse, e = 0, S_in = dS^T, intra = update = scale, inter = 1
// (the sums over s >= t of the backward pass are the forward's sums in reversed time; with e = 0 the state is
// carried with its decay already applied, so neither a division by g nor by scale is needed, and the last
// sweep's S_out is dL/dS_0).
//
// Within a chunk of C rows the sums are matrix products; between chunks only S is carried.
#pragma once

#include "solver.cuh"

namespace pararnn {

struct LaRows {  // a [B, T, heads, width] operand: element strides, innermost contiguous
    const void *p;
    long long sb, st, sh;
    int group;  // head h of the sweep reads operand head h / group
};

struct LaSweep {
    int B, T, H, dk, dv;  // dk: width of a and b; dv: width of c and out
    int dtype;            // of a, b, c
    LaRows a, b, c;
    const float *log_decay;  // [H]
    const int *lengths;      // [B] or null
    const float *s_in;       // [B, H, .] or null (zero); element (i, j) at i * s_i + j * s_j
    float *s_out;            // or null
    int s_i, s_j;
    void *out;  // dense [B, T, H, out_w], out_w >= dv (bf16 sweeps: a multiple of 8)
    int out_w, out_f32;
    int reverse, e;
    float intra, inter, update;
    int n_seg, seg;  // segments of `seg` tokens each (n_seg = 1: the whole sequence)
    float *seg_state;  // [B*H, n_seg, dk, dv]: pass 1 writes each segment's own S_out, the join its S_in
};

// Segments of time: with few sequences and heads the sweep is split into segments that run at once: pass 1
// computes each segment's own state, a join decays and adds them up, pass 2 runs every segment from its start.
struct LaPlan {
    int n_seg, seg;
};
// `sweeps` of them run at once; ragged: the sequences' lengths may differ
LaPlan la_plan(int B, int T, int H, int dk, int dv, int dtype, int sweeps, bool ragged);

// n <= 3 independent sweeps; those that can share a launch do.
cudaError_t launch_la_sweeps(const LaSweep *w, int n, cudaStream_t s);

// bf16 operands on tensor cores: n <= 3 sweeps in one launch, every one of which goes together with the first
cudaError_t launch_la_tc(const LaSweep *w, int n, cudaStream_t s);
bool la_tc_together(const LaSweep &x, const LaSweep &y);
// whether TMA can read the operand: base and strides on 16 bytes, no axis of stride 0
bool la_tc_readable(const LaRows &r, int B, int T, int heads);
// bf16 rows to and from a dense [B, T, heads, width rounded up to 8]
cudaError_t launch_la_pack(const LaRows &src, void *dst, int B, int T, int heads, int width, cudaStream_t s);
cudaError_t launch_la_unpack(const void *src, void *dst, long long rows, int width, cudaStream_t s);

cudaError_t launch_la_join(const LaSweep &w, cudaStream_t s);  // segments' own states -> their start states

cudaError_t launch_la_group_sum(const float *part, void *out, int dtype, long long rows, int Hkv, int per, int d,
                                int dp, cudaStream_t s);

// The single-token step; state row `slots[b]` (or b) of [n_slots, H, dk, dv] belongs to row b.
struct LaStep {
    int B, H, dk, dv, dtype, n_slots;
    LaRows q, k, v;  // st unused
    const float *log_decay, *state;
    const int *slots;
    float scale;
    void *out;  // dense [B, H, dv]
    float *out_state;
};
cudaError_t launch_la_step(const LaStep &w, cudaStream_t s);

// log g, kept finite: exp(n * -1e4) is 0 for every n >= 1 and 1 for n = 0, as g = 0 wants it.
__device__ __forceinline__ float safe_log_decay(float x) { return fmaxf(x, -1e4f); }
// g^n.  n * log g is formed in fp64 so that far positions keep their digits.
__device__ __forceinline__ float decay_pow(float ld, long long n) {
    return expf(static_cast<float>(static_cast<double>(ld) * static_cast<double>(n)));
}
// What decay_pow leaves of g^n.  A weight that the state is multiplied by again and again takes both parts: rounded to
// fp32 it would be another decay, off by as many roundings as there are chunks (memories of 1e5 tokens, 16384 of them:
// 9e-6 of the state)
__device__ __forceinline__ float decay_rest(float ld, long long n) {
    return static_cast<float>(exp(static_cast<double>(ld) * static_cast<double>(n)) - static_cast<double>(decay_pow(ld, n)));
}

}  // namespace pararnn
