// causal_conv.cu -- the short causal convolution over time with one filter per channel, channels last: forward, backward
// and one token at a time (sm_100a).
//
//   p_t = bias + sum_k w_k x_(t-k) with w_k = weight[W-1-k],   y_t = p_t or p_t sigmoid(p_t)
//   q_t = dy_t act'(p_t),   dx_t = sum_k w_k q_(t+k),   dweight[W-1-k] = sum q_t x_(t-k),   dbias = sum q_t
// Inputs before the first are the state's rows, or zero; the last W - 1 inputs are the next state.
#include <algorithm>
#include <type_traits>

#include "causal_conv.cuh"
#include "rows.cuh"
#include "selective_scan.cuh"

namespace pararnn {
using namespace rows;
namespace {

// V neighbouring channels of a token as they lie in memory: V 32-bit words, or V / 2 of them (half a one) in bf16
template <typename T, int V>
struct Raw {
    static constexpr int WORDS = sizeof(T) == 4 ? V : (V + 1) / 2;
    unsigned v[WORDS];
    __device__ __forceinline__ void get(const T *p) {
        if constexpr (sizeof(T) * V == 16) {
            const uint4 q = *reinterpret_cast<const uint4 *>(p);
            v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        } else if constexpr (sizeof(T) * V == 8) {
            const uint2 q = *reinterpret_cast<const uint2 *>(p);
            v[0] = q.x, v[1] = q.y;
        } else if constexpr (sizeof(T) * V == 4) {
            v[0] = *reinterpret_cast<const unsigned *>(p);
        } else {
            v[0] = *reinterpret_cast<const unsigned short *>(p);
        }
    }
    __device__ __forceinline__ void to(float (&f)[V]) const {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            if constexpr (sizeof(T) == 4) f[u] = __uint_as_float(v[u]);
            else f[u] = __uint_as_float(u % 2 == 0 ? v[u / 2] << 16 : v[u / 2] & 0xffff0000u);
        }
    }
};
template <typename T, int V>
__device__ __forceinline__ void put(T *p, const float (&f)[V]) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (V == 4) *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
        else if constexpr (V == 2) *reinterpret_cast<float2 *>(p) = make_float2(f[0], f[1]);
        else *p = f[0];
    } else if constexpr (V == 1) {
        *p = __float2bfloat16(f[0]);
    } else {
        unsigned v[V / 2];
#pragma unroll
        for (int u = 0; u < V; u += 2) {
            const __nv_bfloat162 q = __floats2bfloat162_rn(f[u], f[u + 1]);
            v[u / 2] = *reinterpret_cast<const unsigned *>(&q);
        }
        if constexpr (V == 4) *reinterpret_cast<uint2 *>(p) = make_uint2(v[0], v[1]);
        else *reinterpret_cast<unsigned *>(p) = v[0];
    }
}

// 1 / (1 + exp(-p)) for y.  A bf16 y rounds 2^-9 of the value away: there the exponent need not carry p log2(e)'s last digits.
template <typename T>
__device__ __forceinline__ float sigmoid_t(float p) {
    if constexpr (sizeof(T) == 4) return ss::sigmoid_of(p);
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(p * -kLog2eF));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
template <typename T>
__device__ __forceinline__ float act_of(float p, bool silu) {
    return silu ? p * sigmoid_t<T>(p) : p;
}
// with all digits whatever the type: it goes into dweight and dbias, which are fp32
__device__ __forceinline__ float slope_of(float p, bool silu) {
    if (!silu) return 1.f;
    const float s = ss::sigmoid_of(p);
    return s * fmaf(p, 1.f - s, 1.f);
}

// Where the inputs of one sequence's V channels are.  x_t; before the first token the state's rows; zero elsewhere.
template <typename T, int V>
struct Inputs {
    const T *x, *state;  // x_0; the state's row W - 1, which would be x_0
    long long st, D;
    int len, W;
    __device__ Inputs(const CcArgs &w, int b, int c)
        : x(static_cast<const T *>(w.x.p) + b * w.x.sb + c),
          state(w.state == nullptr ? nullptr
                                   : static_cast<const T *>(w.state) + (static_cast<long long>(b) * (w.W - 1) + w.W - 1) * w.D + c),
          st(w.x.st), D(w.D), len(count(w.lengths, b, w.T)), W(w.W) {}
    __device__ __forceinline__ Raw<T, V> later(long long t) const {  // t >= 0
        Raw<T, V> r{};
        if (t < len) r.get(x + t * st);
        return r;
    }
    __device__ __forceinline__ Raw<T, V> at(long long t) const {
        if (t >= 0) return later(t);
        Raw<T, V> r{};
        if (state != nullptr && t >= 1 - W) r.get(state + t * D);
        return r;
    }
};

template <int W, int V>
__device__ __forceinline__ void load_filter(const CcArgs &w, int c, float (&wk)[W][V], float (&bias)[V]) {
    const float *p = w.weight + static_cast<long long>(c) * W;
    float f[V * W];
    if constexpr (V == 4) {  // the four filters lie one after the other
        if (reinterpret_cast<uintptr_t>(w.weight) % 16 == 0) {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float4 q = reinterpret_cast<const float4 *>(p)[i];
                f[4 * i] = q.x, f[4 * i + 1] = q.y, f[4 * i + 2] = q.z, f[4 * i + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V * W; ++i) f[i] = p[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V * W; ++i) f[i] = p[i];
    }
#pragma unroll
    for (int u = 0; u < V; ++u) {
#pragma unroll
        for (int k = 0; k < W; ++k) wk[k][u] = f[u * W + W - 1 - k];
        bias[u] = w.bias != nullptr ? w.bias[c + u] : 0.f;
    }
}
// p of a token from the window win[k] = x_(t-k), two channels in an operation
template <int W, int V>
__device__ __forceinline__ void pre(const float (&wk)[W][V], const float (&bias)[V], const float (&win)[W][V], float (&p)[V]) {
    if constexpr (V == 1) {
        p[0] = bias[0];
#pragma unroll
        for (int k = W - 1; k >= 0; --k) p[0] = fmaf(wk[k][0], win[k][0], p[0]);
    } else {
#pragma unroll
        for (int u = 0; u < V; u += 2) {
            u64 s = pk(bias[u], bias[u + 1]);
#pragma unroll
            for (int k = W - 1; k >= 0; --k) s = fma2(pk(wk[k][u], wk[k][u + 1]), pk(win[k][u], win[k][u + 1]), s);
            upk(s, p[u], p[u + 1]);
        }
    }
}
// c += a b
template <int V>
__device__ __forceinline__ void add_product(const float (&a)[V], const float (&b)[V], float (&c)[V]) {
    if constexpr (V == 1) {
        c[0] = fmaf(a[0], b[0], c[0]);
    } else {
#pragma unroll
        for (int u = 0; u < V; u += 2) upk(fma2(pk(a[u], a[u + 1]), pk(b[u], b[u + 1]), pk(c[u], c[u + 1])), c[u], c[u + 1]);
    }
}
template <int W, int V>
__device__ __forceinline__ void shift(float (&win)[W][V], const float (&x)[V]) {
#pragma unroll
    for (int k = W - 1; k > 0; --k)
#pragma unroll
        for (int u = 0; u < V; ++u) win[k][u] = win[k - 1][u];
#pragma unroll
    for (int u = 0; u < V; ++u) win[0][u] = x[u];
}

// A thread takes V channels (four where they are aligned) through `run` tokens with the last W inputs in registers and the
// next tokens' loads on their way; consecutive threads take consecutive channels.
// 8 x 4096 x 4096 in bf16 with SiLU 120 us, 0.68 of HBM's rate, with issue slots 65 % and the MUFU pipe 51 % busy at 34 % of the
// warps (eight channels to a thread: 311, one CTA to an SM; eight tokens ahead: 132).
template <typename T, int W, int V>
__global__ void __launch_bounds__(256, W <= 4 ? 3 : 2) cc_forward_kernel(const CcArgs w, int run) {
    const int nv = w.D / V, runs = (w.T + run - 1) / run;
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= static_cast<long long>(nv) * runs * w.B) return;
    const int c = static_cast<int>(i % nv) * V, r = static_cast<int>(i / nv % runs), b = static_cast<int>(i / nv / runs);
    const Inputs<T, V> in(w, b, c);
    const int t0 = r * run, t_end = min(w.T, t0 + run);
    const bool silu = w.act == PARARNN_ACT_SILU;
    constexpr int AHEAD = 4;
    Raw<T, V> next[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) next[j] = in.later(t0 + j);
    float wk[W][V], bias[V], win[W][V], x[V];
    load_filter(w, c, wk, bias);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) in.at(t0 - 1 - k).to(win[k]);
    T *y = static_cast<T *>(w.y) + (static_cast<long long>(b) * w.T + t0) * w.D + c;
    for (int t = t0; t < t_end; t += AHEAD) {
        Raw<T, V> now[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) now[j] = next[j];
        if (t + AHEAD < t_end) {
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) next[j] = in.later(t + AHEAD + j);
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            now[j].to(x);
            shift(win, x);
            float p[V];
            pre(wk, bias, win, p);
            const bool on = t + j < in.len;
#pragma unroll
            for (int u = 0; u < V; ++u) p[u] = on ? act_of<T>(p[u], silu) : 0.f;
            if (t + j < t_end) put<T, V>(y, p);
            y += w.D;
        }
    }
    if (r == 0) {
        T *last = static_cast<T *>(w.last) + static_cast<long long>(b) * (W - 1) * w.D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            in.at(static_cast<long long>(in.len) - (W - 1) + j).to(x);
            put<T, V>(last + static_cast<long long>(j) * w.D, x);
        }
    }
}

// The same walk for dx, W - 1 tokens behind p; a CTA is tx vectors of channels by 256 / tx runs, and keeps its sums for the
// parameters over all the runs it takes.  8 x 4096 x 2048 in bf16, 4 taps: 122 us, 0.50 of HBM's rate: 37 instructions to an
// element in 60 % of the issue slots, at 23 % of the warps (four channels to a thread, checks at every token or runs of 32 took
// 1.4 to 1.5 times as long).
template <typename T, int W, int V>
__global__ void __launch_bounds__(256, 2) cc_backward_kernel(const CcArgs w, int tx, int run) {
    extern __shared__ float s_part[];  // [V (W + 1)][256]
    const int x_of = threadIdx.x % tx, y_of = threadIdx.x / tx, ty = 256 / tx;
    const int c = (blockIdx.x * tx + x_of) * V;
    const int runs = (w.T + run - 1) / run;
    const long long all = static_cast<long long>(runs) * w.B;
    const bool silu = w.act == PARARNN_ACT_SILU, on = c < w.D;
    float wk[W][V] = {}, bias[V] = {}, dw[W][V] = {}, db[V] = {};
    // the sums so far, of sums over 64 tokens: one long chain would lose digits
    auto add_up = [&](bool first) {
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
            for (int k = 0; k <= W; ++k) {
                float &part = s_part[(u * (W + 1) + k) * 256 + threadIdx.x], &own = k < W ? dw[W - 1 - k][u] : db[u];
                part = first ? own : part + own;
                own = 0.f;
            }
    };
    add_up(true);
    if (on) {
        load_filter(w, c, wk, bias);
        for (long long i = static_cast<long long>(blockIdx.y) * ty + y_of; i < all; i += static_cast<long long>(gridDim.y) * ty) {
            const int r = static_cast<int>(i % runs), b = static_cast<int>(i / runs);
            const Inputs<T, V> in(w, b, c);
            const int t0 = r * run, t_end = min(w.T, t0 + run), len = in.len;
            const int from = r == 0 ? 1 - W : t0;  // of dx, the state's rows among it
            const T *pdy = static_cast<const T *>(w.dy.p) + b * w.dy.sb + c;
            auto grad = [&](int t) {
                Raw<T, V> g{};
                if (t < len) g.get(pdy + t * w.dy.st);
                return g;
            };
            constexpr int AHEAD = 4;
            Raw<T, V> nx[AHEAD], ng[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) nx[j] = in.later(t0 + j), ng[j] = grad(t0 + j);
            float win[W][V] = {}, q[W][V] = {}, x[V], g[V];  // win[k]: x_(t-k); q[k]: q_(t-k)
#pragma unroll
            for (int k = 0; k < W - 1; ++k) in.at(t0 - 1 - k).to(win[k]);
            // token `at`: its q, and dx of token at - (W - 1), which is complete with it; own: not one behind the run
            T *dx = static_cast<T *>(w.dx) + (static_cast<long long>(b) * w.T + t0 - (W - 1)) * w.D + c;
            const int plain = max(len - W, -1) + 1;  // dx of tokens 0 .. plain - 1 has no part of dlast and counts
            auto token = [&](auto inside, int at, bool own, const Raw<T, V> &rx, const Raw<T, V> &rg) {
                rx.to(x), rg.to(g);
                shift(win, x);
                float p[V], out[V] = {};
                pre(wk, bias, win, p);
#pragma unroll
                for (int u = 0; u < V; ++u) p[u] = g[u] * slope_of(p[u], silu);  // g is zero behind the sequence
                shift(q, p);
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    if (!own) p[u] = 0.f;
                    db[u] += p[u];
                }
#pragma unroll
                for (int k = 0; k < W; ++k) {
                    add_product(p, win[k], dw[k]);
                    add_product(wk[W - 1 - k], q[k], out);
                }
                const int back = at - (W - 1);
                if constexpr (decltype(inside)::value) {
                    put<T, V>(dx, out);
                } else if (back >= from && back < t_end) {
                    if (static_cast<unsigned>(back) >= static_cast<unsigned>(plain)) {
                        const int j_last = back - len + W - 1;  // the row of dlast that is x_back
                        if (w.dlast != nullptr && j_last >= 0 && j_last < W - 1) {
                            Raw<T, V> l;
                            l.get(static_cast<const T *>(w.dlast) + (static_cast<long long>(b) * (W - 1) + j_last) * w.D + c);
                            l.to(x);
#pragma unroll
                            for (int u = 0; u < V; ++u) out[u] += x[u];
                        }
                        if (back >= len) {
#pragma unroll
                            for (int u = 0; u < V; ++u) out[u] = 0.f;
                        }
                    }
                    if (back >= 0) put<T, V>(dx, out);
                    else if (w.dstate != nullptr)
                        put<T, V>(static_cast<T *>(w.dstate) + (static_cast<long long>(b) * (W - 1) + back + W - 1) * w.D + c, out);
                }
                dx += w.D;
            };
            const int stop = t_end + W - 1;
            const T *px = in.x + static_cast<long long>(t0 + AHEAD) * in.st, *pg = pdy + static_cast<long long>(t0 + AHEAD) * w.dy.st;
            for (int t = t0; t < stop; add_up(false)) {
                do {
                    Raw<T, V> cx[AHEAD], cg[AHEAD];
#pragma unroll
                    for (int j = 0; j < AHEAD; ++j) cx[j] = nx[j], cg[j] = ng[j];
                    if (t + 2 * AHEAD <= len) {
#pragma unroll
                        for (int j = 0; j < AHEAD; ++j) nx[j].get(px + j * w.x.st), ng[j].get(pg + j * w.dy.st);
                    } else if (t + AHEAD < stop) {
#pragma unroll
                        for (int j = 0; j < AHEAD; ++j) nx[j] = in.later(t + AHEAD + j), ng[j] = grad(t + AHEAD + j);
                    }
                    px += AHEAD * w.x.st, pg += AHEAD * w.dy.st;
                    // inside a run nothing has to be asked: dx is of its own tokens, which count and have no part of dlast
                    if (t >= t0 + W - 1 && t + AHEAD <= t_end && t + AHEAD - W < plain) {
#pragma unroll
                        for (int j = 0; j < AHEAD; ++j) token(std::true_type{}, t + j, true, cx[j], cg[j]);
                    } else {
#pragma unroll
                        for (int j = 0; j < AHEAD; ++j) token(std::false_type{}, t + j, t + j < t_end, cx[j], cg[j]);
                    }
                    t += AHEAD;
                } while (t < stop && (t - t0 & 63) != 0);
            }
        }
    }
    // the CTA's sums, over its rows of threads in order
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
            for (int u = 0; u < V; ++u) p[u] = act_of<T>(p[u], silu);
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
// rows whose vectors of v channels start on their own alignment
bool rows_on(const CcRows &r, int dtype, int v) {
    return reinterpret_cast<uintptr_t>(r.p) % (v * esize(dtype)) == 0 && r.sb % v == 0 && r.st % v == 0;
}

// Tokens of a thread: long runs read less of their neighbours, short ones fill the card (two waves of 2048 threads per SM)
int run_of(const CcArgs &a, int v) {
    const long long at_64 = static_cast<long long>(a.D / v) * a.B * ((a.T + 63) / 64);
    for (int run = 64; run > 8; run /= 2)
        if (at_64 * (64 / run) >= 148 * 4096) return run;
    return 8;
}
template <typename T, int W>
void forward_of(const CcArgs &a, bool vec, cudaStream_t s) {
    const int v = vec ? 4 : 1, run = run_of(a, v);
    const long long n = static_cast<long long>(a.D / v) * ((a.T + run - 1) / run) * a.B;
    const unsigned grid = static_cast<unsigned>((n + 255) / 256);
    if (vec) cc_forward_kernel<T, W, 4><<<grid, 256, 0, s>>>(a, run);
    else cc_forward_kernel<T, W, 1><<<grid, 256, 0, s>>>(a, run);
}
struct Grid {
    int tx, x, y, run;
};
Grid backward_grid(const CcArgs &a, int v) {
    const int nv = (a.D + v - 1) / v;
    int tx = 1;
    while (tx < nv && tx < 32) tx *= 2;
    // one wave of two CTAs per SM, and a run for each of their threads: every run's start waits for its first loads
    const int x = (nv + tx - 1) / tx, ty = 256 / tx, rows = std::max(1, 148 * 2 / x) * ty;
    const int splits = std::max(1, rows / a.B);
    const int run = std::max(8, ((a.T + splits - 1) / splits + 3) / 4 * 4);
    const long long all = static_cast<long long>((a.T + run - 1) / run) * a.B;
    return {tx, x, static_cast<int>(std::min<long long>((all + ty - 1) / ty, rows / ty)), run};
}
template <typename T, int W>
void backward_of(const CcArgs &a, bool vec, cudaStream_t s) {
    const Grid g = backward_grid(a, vec ? 2 : 1);
    const dim3 grid(g.x, g.y);
    if (vec) cc_backward_kernel<T, W, 2><<<grid, 256, 256 * 2 * (W + 1) * sizeof(float), s>>>(a, g.tx, g.run);
    else cc_backward_kernel<T, W, 1><<<grid, 256, 256 * (W + 1) * sizeof(float), s>>>(a, g.tx, g.run);
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
    return std::max(backward_grid(a, 1).y, a.D % 2 == 0 ? backward_grid(a, 2).y : 1);
}

cudaError_t launch_cc_forward(const CcArgs &a, cudaStream_t s) {
    const bool vec = a.D % 4 == 0 && rows_on(a.x, a.dtype, 4) && on16(a.state) && on16(a.y) && on16(a.last);
    if (a.dtype == PARARNN_F32) launch_width<float>(a, false, vec, s);
    else launch_width<__nv_bfloat16>(a, false, vec, s);
    return cudaGetLastError();
}

cudaError_t launch_cc_backward(const CcArgs &a, cudaStream_t s) {
    const bool vec = a.D % 2 == 0 && rows_on(a.x, a.dtype, 2) && rows_on(a.dy, a.dtype, 2) && on16(a.state) && on16(a.dlast);
    if (a.dtype == PARARNN_F32) launch_width<float>(a, true, vec, s);
    else launch_width<__nv_bfloat16>(a, true, vec, s);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long n = static_cast<long long>(a.D) * a.W;
    return launch_rows_sum({a.part, backward_grid(a, vec ? 2 : 1).y, n + a.D, {a.dweight, a.dbias, nullptr}, {n, a.D, 0}}, s);
}

cudaError_t launch_cc_step(const CcStep &w, cudaStream_t s) {
    const bool vec = w.D % 4 == 0 && rows_on(w.x, w.dtype, 4);
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
