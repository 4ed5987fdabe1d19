// causal_conv.cu -- the short causal convolution over time with one filter per channel, channels last: forward, backward
// and one token at a time (sm_100a).
//
//   p_t = bias + sum_k w_k x_(t-k) with w_k = weight[W-1-k],   y_t = p_t or p_t sigmoid(p_t)
//   q_t = dy_t act'(p_t),   dx_t = sum_k w_k q_(t+k),   dweight[W-1-k] = sum q_t x_(t-k),   dbias = sum q_t
// Inputs before the first are the state's rows, or zero; the last W - 1 inputs are the next state.
#include <algorithm>

#include "causal_conv.cuh"
#include "rows.cuh"

namespace pararnn {
using namespace rows;
namespace {

__device__ __forceinline__ float act_of(float p, bool silu) {
    return silu ? p * __fdividef(1.f, 1.f + expf(-p)) : p;
}
__device__ __forceinline__ float slope_of(float p, bool silu) {
    if (!silu) return 1.f;
    const float s = __fdividef(1.f, 1.f + expf(-p));
    return s * fmaf(p, 1.f - s, 1.f);
}

// x_t of V channels from c on; before the first token the state's rows
template <typename T, int V>
__device__ __forceinline__ void input(const CcArgs &w, int b, long long t, int c, int len, float (&v)[V]) {
#pragma unroll
    for (int u = 0; u < V; ++u) v[u] = 0.f;
    if (t >= 0) {
        if (t < len) load<V>(static_cast<const T *>(w.x.p) + b * w.x.sb + t * w.x.st + c, v);
    } else if (w.state != nullptr && t >= 1 - w.W) {
        load<V>(static_cast<const T *>(w.state) + (static_cast<long long>(b) * (w.W - 1) + t + w.W - 1) * w.D + c, v);
    }
}

constexpr int kRun = 32;  // tokens of a thread

// A thread takes V channels through kRun tokens with the last W inputs in registers; consecutive threads take consecutive
// channels.  Bound by HBM.
template <typename T, int W, int V>
__global__ void __launch_bounds__(256) cc_forward_kernel(const CcArgs w) {
    const int nv = w.D / V, runs = (w.T + kRun - 1) / kRun;
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= static_cast<long long>(nv) * runs * w.B) return;
    const int c = static_cast<int>(i % nv) * V, run = static_cast<int>(i / nv % runs), b = static_cast<int>(i / nv / runs);
    const int len = count(w.lengths, b, w.T), t0 = run * kRun, t_end = min(w.T, t0 + kRun);
    const bool silu = w.act == PARARNN_ACT_SILU;
    float wk[W][V], bias[V] = {}, win[W][V];  // win[k]: x_(t-k)
#pragma unroll
    for (int u = 0; u < V; ++u) {
#pragma unroll
        for (int k = 0; k < W; ++k) wk[k][u] = w.weight[static_cast<long long>(c + u) * W + W - 1 - k];
        if (w.bias != nullptr) bias[u] = w.bias[c + u];
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) input<T, V>(w, b, t0 - 1 - k, c, len, win[k]);
    T *y = static_cast<T *>(w.y) + static_cast<long long>(b) * w.T * w.D + c;
    constexpr int AHEAD = 8;
    for (int t = t0; t < t_end; t += AHEAD) {
        float x[AHEAD][V];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) input<T, V>(w, b, t + j, c, len, x[j]);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
#pragma unroll
            for (int k = W - 1; k > 0; --k)
#pragma unroll
                for (int u = 0; u < V; ++u) win[k][u] = win[k - 1][u];
            float out[V];
#pragma unroll
            for (int u = 0; u < V; ++u) {
                win[0][u] = x[j][u];
                float p = bias[u];
#pragma unroll
                for (int k = W - 1; k >= 0; --k) p = fmaf(wk[k][u], win[k][u], p);
                out[u] = t + j < len ? act_of(p, silu) : 0.f;
            }
            if (t + j < t_end) store<V>(y + static_cast<long long>(t + j) * w.D, out);
        }
    }
    if (run == 0) {
        T *last = static_cast<T *>(w.last) + static_cast<long long>(b) * (W - 1) * w.D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            float x[V];
            input<T, V>(w, b, static_cast<long long>(len) - (W - 1) + j, c, len, x);
            store<V>(last + static_cast<long long>(j) * w.D, x);
        }
    }
}

// The same walk for dx, W - 1 tokens behind p; a CTA is tx vectors of channels by 256 / tx runs, and keeps its sums for the
// parameters in registers over all the runs it takes.
template <typename T, int W, int V>
__global__ void __launch_bounds__(256) cc_backward_kernel(const CcArgs w, int tx) {
    extern __shared__ float s_part[];  // [256][V (W + 1)] turned to [V (W + 1)][256]
    const int x_of = threadIdx.x % tx, y_of = threadIdx.x / tx, ty = 256 / tx;
    const int c = (blockIdx.x * tx + x_of) * V;
    const int runs = (w.T + kRun - 1) / kRun;
    const long long all = static_cast<long long>(runs) * w.B;
    const bool silu = w.act == PARARNN_ACT_SILU, on = c < w.D;
    float wk[W][V] = {}, bias[V] = {}, dw[W][V] = {}, db[V] = {};
    if (on) {
#pragma unroll
        for (int u = 0; u < V; ++u) {
#pragma unroll
            for (int k = 0; k < W; ++k) wk[k][u] = w.weight[static_cast<long long>(c + u) * W + W - 1 - k];
            if (w.bias != nullptr) bias[u] = w.bias[c + u];
        }
        for (long long i = static_cast<long long>(blockIdx.y) * ty + y_of; i < all; i += static_cast<long long>(gridDim.y) * ty) {
            const int run = static_cast<int>(i % runs), b = static_cast<int>(i / runs);
            const int len = count(w.lengths, b, w.T), t0 = run * kRun, t_end = min(w.T, t0 + kRun);
            const int from = run == 0 ? 1 - W : t0;  // of dx, the state's rows among it
            float win[W][V] = {}, q[W][V] = {};       // win[k]: x_(t-k); q[k]: q_(t-k)
            // x before the first q that is needed: of token max(from, 0)
#pragma unroll
            for (int k = 0; k < W - 1; ++k) input<T, V>(w, b, max(from, 0) - 1 - k, c, len, win[k]);
            const T *pdy = static_cast<const T *>(w.dy.p) + b * w.dy.sb + c;
            constexpr int AHEAD = 4;
            for (int t = max(from, 0); t < t_end + W - 1; t += AHEAD) {
                float x[AHEAD][V], g[AHEAD][V];
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    input<T, V>(w, b, t + j, c, len, x[j]);
#pragma unroll
                    for (int u = 0; u < V; ++u) g[j][u] = 0.f;
                    if (t + j < len) load<V>(pdy + (t + j) * w.dy.st, g[j]);
                }
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    const int at = t + j, back = at - (W - 1);  // dx that is complete with q_at
#pragma unroll
                    for (int k = W - 1; k > 0; --k)
#pragma unroll
                        for (int u = 0; u < V; ++u) win[k][u] = win[k - 1][u], q[k][u] = q[k - 1][u];
                    float out[V];
#pragma unroll
                    for (int u = 0; u < V; ++u) {
                        win[0][u] = x[j][u];
                        float p = bias[u];
#pragma unroll
                        for (int k = W - 1; k >= 0; --k) p = fmaf(wk[k][u], win[k][u], p);
                        q[0][u] = at < len ? g[j][u] * slope_of(p, silu) : 0.f;
                        const float own = at < t_end ? q[0][u] : 0.f;
                        db[u] += own;
                        float sum = 0.f;
#pragma unroll
                        for (int k = 0; k < W; ++k) {
                            dw[k][u] = fmaf(own, win[k][u], dw[k][u]);
                            sum = fmaf(wk[W - 1 - k][u], q[k][u], sum);
                        }
                        out[u] = sum;
                    }
                    if (back >= from && back < t_end) {
                        const int j_last = back - len + W - 1;  // the row of dlast that is x_back
                        if (w.dlast != nullptr && j_last >= 0 && j_last < W - 1) {
                            float l[V];
                            load<V>(static_cast<const T *>(w.dlast) + (static_cast<long long>(b) * (W - 1) + j_last) * w.D + c, l);
#pragma unroll
                            for (int u = 0; u < V; ++u) out[u] += l[u];
                        }
                        if (back >= 0) {
                            if (back >= len) {
#pragma unroll
                                for (int u = 0; u < V; ++u) out[u] = 0.f;
                            }
                            store<V>(static_cast<T *>(w.dx) + (static_cast<long long>(b) * w.T + back) * w.D + c, out);
                        } else if (w.dstate != nullptr) {
                            store<V>(static_cast<T *>(w.dstate) + (static_cast<long long>(b) * (W - 1) + back + W - 1) * w.D + c, out);
                        }
                    }
                }
            }
        }
    }
    // the CTA's sums, over its rows of threads in order
#pragma unroll
    for (int u = 0; u < V; ++u) {
#pragma unroll
        for (int k = 0; k < W; ++k) s_part[(u * (W + 1) + W - 1 - k) * 256 + threadIdx.x] = dw[k][u];
        s_part[(u * (W + 1) + W) * 256 + threadIdx.x] = db[u];
    }
    __syncthreads();
    for (int o = threadIdx.x; o < tx * V * (W + 1); o += 256) {
        const int k = o / tx, xx = o % tx, u = k / (W + 1);
        const int channel = (blockIdx.x * tx + xx) * V + u;
        if (channel >= w.D) continue;
        float sum = 0.f;
        for (int y = 0; y < ty; ++y) sum += s_part[k * 256 + y * tx + xx];
        const int tap = k % (W + 1);
        float *row = w.part + static_cast<long long>(blockIdx.y) * w.D * (W + 1);
        row[tap < W ? static_cast<long long>(channel) * W + tap : static_cast<long long>(w.D) * W + channel] = sum;
    }
}

// One token of every row: y and the state's rows moved up by one.  Rows that name the same slot are taken in row order by
// the first one's CTA, as tokens that follow each other.
template <typename T, int V>
__global__ void __launch_bounds__(128) cc_step_kernel(const CcStep w) {
    __shared__ int next;
    const int nv = w.D / V, tiles = (nv + 127) / 128, tid = threadIdx.x;
    int b = blockIdx.x / tiles;
    const int c = (blockIdx.x % tiles * 128 + tid) * V;
    const bool on = c < w.D;
    T *py = static_cast<T *>(w.y);
    const int slot = w.slots == nullptr ? b : w.slots[b];
    if (slot < 0 || slot >= w.n_slots) {  // no state behind this row
        const float zero[V] = {};
        if (on) store<V>(py + static_cast<long long>(b) * w.D + c, zero);
        return;
    }
    if (w.slots != nullptr) {
        int earlier = 0;
        for (int i = tid; i < b; i += 128) earlier |= w.slots[i] == slot;
        if (__syncthreads_or(earlier)) return;
    }
    const bool silu = w.act == PARARNN_ACT_SILU;
    const long long at = static_cast<long long>(slot) * (w.W - 1) * w.D + c;
    const T *src = static_cast<const T *>(w.state) + at;
    T *dst = static_cast<T *>(w.out_state) + at;
    while (true) {
        if (w.slots != nullptr) {
            if (tid == 0) next = w.B;
            __syncthreads();
        }
        if (on) {
            float p[V] = {}, x[V];
            if (w.bias != nullptr)
#pragma unroll
                for (int u = 0; u < V; ++u) p[u] = w.bias[c + u];
            for (int j = 0; j < w.W; ++j) {
                if (j < w.W - 1) load<V>(src + static_cast<long long>(j) * w.D, x);
                else load<V>(static_cast<const T *>(w.x.p) + b * w.x.sb + c, x);
#pragma unroll
                for (int u = 0; u < V; ++u) p[u] = fmaf(w.weight[static_cast<long long>(c + u) * w.W + j], x[u], p[u]);
                if (j > 0) store<V>(dst + static_cast<long long>(j - 1) * w.D, x);
            }
#pragma unroll
            for (int u = 0; u < V; ++u) p[u] = act_of(p[u], silu);
            store<V>(py + static_cast<long long>(b) * w.D + c, p);
        }
        if (w.slots == nullptr) return;
        for (int i = b + 1 + tid; i < w.B; i += 128)
            if (w.slots[i] == slot) {
                atomicMin(&next, i);
                break;
            }
        __syncthreads();
        b = next;
        if (b >= w.B) return;
        src = dst;  // each thread reads back what it wrote itself
        __syncthreads();
    }
}

size_t esize(int dtype) { return dtype == PARARNN_F32 ? 4 : 2; }
bool on16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
// rows whose vectors of four start on their own alignment
bool rows4(const CcRows &r, int dtype) {
    return reinterpret_cast<uintptr_t>(r.p) % (4 * esize(dtype)) == 0 && r.sb % 4 == 0 && r.st % 4 == 0;
}

template <typename T, int W>
void forward_of(const CcArgs &a, bool vec, cudaStream_t s) {
    const long long n = static_cast<long long>(a.D / (vec ? 4 : 1)) * ((a.T + kRun - 1) / kRun) * a.B;
    const unsigned grid = static_cast<unsigned>((n + 255) / 256);
    if (vec) cc_forward_kernel<T, W, 4><<<grid, 256, 0, s>>>(a);
    else cc_forward_kernel<T, W, 1><<<grid, 256, 0, s>>>(a);
}
struct Grid {
    int tx, x, y;
};
Grid backward_grid(const CcArgs &a, int v) {
    const int nv = (a.D + v - 1) / v;
    int tx = 1;
    while (tx < nv && tx < 32) tx *= 2;
    const int x = (nv + tx - 1) / tx, ty = 256 / tx;
    const long long all = static_cast<long long>((a.T + kRun - 1) / kRun) * a.B;
    const long long y = std::min<long long>((all + ty - 1) / ty, std::max(1, (148 * 4 + x - 1) / x));
    return {tx, x, static_cast<int>(y)};
}
template <typename T, int W>
void backward_of(const CcArgs &a, bool vec, cudaStream_t s) {
    const Grid g = backward_grid(a, vec ? 4 : 1);
    const dim3 grid(g.x, g.y);
    if (vec) cc_backward_kernel<T, W, 4><<<grid, 256, 256 * 4 * (W + 1) * sizeof(float), s>>>(a, g.tx);
    else cc_backward_kernel<T, W, 1><<<grid, 256, 256 * (W + 1) * sizeof(float), s>>>(a, g.tx);
}

template <typename T, int W>
void launch(const CcArgs &a, bool back, bool vec, cudaStream_t s) {
    if (back) backward_of<T, W>(a, vec, s);
    else forward_of<T, W>(a, vec, s);
}
template <typename T>
void launch_width(const CcArgs &a, bool back, bool vec, cudaStream_t s) {
    switch (a.W) {
        case 2: return launch<T, 2>(a, back, vec, s);
        case 3: return launch<T, 3>(a, back, vec, s);
        case 4: return launch<T, 4>(a, back, vec, s);
        case 5: return launch<T, 5>(a, back, vec, s);
        case 6: return launch<T, 6>(a, back, vec, s);
        case 7: return launch<T, 7>(a, back, vec, s);
        default: return launch<T, 8>(a, back, vec, s);
    }
}

}  // namespace

int cc_backward_rows(const CcArgs &a) {
    return std::max(backward_grid(a, 1).y, a.D % 4 == 0 ? backward_grid(a, 4).y : 1);
}

cudaError_t launch_cc_forward(const CcArgs &a, cudaStream_t s) {
    const bool vec = a.D % 4 == 0 && rows4(a.x, a.dtype) && on16(a.state) && on16(a.y) && on16(a.last);
    if (a.dtype == PARARNN_F32) launch_width<float>(a, false, vec, s);
    else launch_width<__nv_bfloat16>(a, false, vec, s);
    return cudaGetLastError();
}

cudaError_t launch_cc_backward(const CcArgs &a, cudaStream_t s) {
    const bool vec = a.D % 4 == 0 && rows4(a.x, a.dtype) && rows4(a.dy, a.dtype) && on16(a.state) && on16(a.dlast);
    if (a.dtype == PARARNN_F32) launch_width<float>(a, true, vec, s);
    else launch_width<__nv_bfloat16>(a, true, vec, s);
    cudaError_t e = cudaGetLastError();
    const long long n = static_cast<long long>(a.D) * a.W, stride = n + a.D;
    const int parts = backward_grid(a, vec ? 4 : 1).y;
    if (e == cudaSuccess) e = launch_rows_sum(a.part, a.dweight, parts, n, stride, s);
    if (e == cudaSuccess) e = launch_rows_sum(a.part + n, a.dbias, parts, a.D, stride, s);
    return e;
}

cudaError_t launch_cc_step(const CcStep &w, cudaStream_t s) {
    const bool vec = w.D % 4 == 0 && rows4(w.x, w.dtype);
    const int nv = w.D / (vec ? 4 : 1);
    const unsigned grid = static_cast<unsigned>((nv + 127) / 128) * w.B;
    if (w.dtype == PARARNN_F32) {
        if (vec) cc_step_kernel<float, 4><<<grid, 128, 0, s>>>(w);
        else cc_step_kernel<float, 1><<<grid, 128, 0, s>>>(w);
    } else {
        if (vec) cc_step_kernel<__nv_bfloat16, 4><<<grid, 128, 0, s>>>(w);
        else cc_step_kernel<__nv_bfloat16, 1><<<grid, 128, 0, s>>>(w);
    }
    return cudaGetLastError();
}

}  // namespace pararnn
