// group_norm.cu -- group norm with an activation or a gate, channels last, forward and backward (sm_100a).
//
//   z = (x - m) r w + b with m, r = mean and 1 / sqrt(var + eps) of (n, group) over its rows and channels;
//   y = act(z), or z * act(gate).   Backward, with xhat = (x - m) r and n_g elements in a group:
//   dz = dy act'(z) or dy act(gate),  dgate = dy z act'(gate),  db = sum dz,  dw = sum dz xhat,
//   dx = r (w dz - sum_g(w dz) / n_g - xhat sum_g(w dz xhat) / n_g).
//
// Two regimes.  One row per statistic (S = 1, groups of up to 1024 channels: each token's heads): a team of 1 to
// 32 lanes holds a group in registers, so x is read once.  Otherwise (statistics over a sequence): partial
// statistics per block of rows, a join, and a second pass over x that applies them.  All sums are fp32: means
// and squared deviations are formed about a local mean and joined by the pairwise update of Chan, Golub and
// LeVeque (1979), so a large common offset costs no digits; sums are taken in a fixed order.
#include <cuda_bf16.h>

#include "group_norm.cuh"

namespace pararnn {
namespace {

constexpr int kThr = 256;

template <typename T>
__device__ __forceinline__ float ld1(const T *p);
template <>
__device__ __forceinline__ float ld1<float>(const float *p) { return *p; }
template <>
__device__ __forceinline__ float ld1<__nv_bfloat16>(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

template <int V>
__device__ __forceinline__ void load(const float *p, float (&v)[V]) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(p + i);
            v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = p[i];
    }
}
__device__ __forceinline__ void unpack(unsigned u, float &a, float &b) {
    a = __uint_as_float(u << 16);
    b = __uint_as_float(u & 0xffff0000u);
}
template <int V>
__device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&v)[V]) {
    if constexpr (V == 8) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        unpack(u.x, v[0], v[1]), unpack(u.y, v[2], v[3]), unpack(u.z, v[4], v[5]), unpack(u.w, v[6], v[7]);
    } else if constexpr (V == 4) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        unpack(u.x, v[0], v[1]), unpack(u.y, v[2], v[3]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = __bfloat162float(p[i]);
    }
}
template <int V>
__device__ __forceinline__ void store(float *p, const float (&v)[V]) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = v[i];
    }
}
__device__ __forceinline__ unsigned pack(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const unsigned *>(&p);
}
template <int V>
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[V]) {
    if constexpr (V == 8) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7]));
    } else if constexpr (V == 4) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack(v[0], v[1]), pack(v[2], v[3]));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = __float2bfloat16(v[i]);
    }
}

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + expf(-z)); }
// act(z) and act'(z)
__device__ __forceinline__ float act_of(float z, int act) {
    if (act == PARARNN_ACT_SILU) return z * sigmoid(z);
    if (act == PARARNN_ACT_GELU) return z * normcdff(z);
    return z;
}
__device__ __forceinline__ float act_slope(float z, int act) {
    if (act == PARARNN_ACT_SILU) {
        const float s = sigmoid(z);
        return s * fmaf(z, 1.f - s, 1.f);
    }
    if (act == PARARNN_ACT_GELU) return fmaf(z * 0.3989422804014327f, expf(-0.5f * z * z), normcdff(z));
    return 1.f;
}

// (count, mean, sum of squared deviations) of two disjoint sets, joined
struct Moments {
    float n, mean, m2;
};
__device__ __forceinline__ Moments join(const Moments &a, const Moments &b) {
    const float n = a.n + b.n;
    if (b.n == 0.f) return a;
    if (a.n == 0.f) return b;
    const float d = b.mean - a.mean, f = b.n / n;
    return {n, fmaf(d, f, a.mean), a.m2 + b.m2 + d * d * a.n * f};
}
__device__ __forceinline__ Moments shuffle_xor(const Moments &a, int m) {
    return {__shfl_xor_sync(~0u, a.n, m), __shfl_xor_sync(~0u, a.mean, m), __shfl_xor_sync(~0u, a.m2, m)};
}

__device__ __forceinline__ int row_count(const GnArgs &a, int n) {
    if (a.lengths == nullptr) return a.S;
    const int c = a.lengths[n];
    return c < 0 ? 0 : (c > a.S ? a.S : c);
}

template <int V>
__device__ __forceinline__ void load_wb(const GnArgs &a, int c, float (&w)[V], float (&b)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = 1.f, b[i] = 0.f;
    if (a.weight != nullptr) load<V>(a.weight + c, w);
    if (a.bias != nullptr) load<V>(a.bias + c, b);
}

// ---- one row per statistic ----------------------------------------------------------------------------------

// Teams of TL lanes; a lane holds K vectors of V channels of its group: channels (k TL + lane) V + i.
// A team keeps its group and walks the rows, so weights (and, backward, their gradients) stay in registers.
struct RowPlan {
    int team;        // lanes per group, a power of two
    int grid;        // CTAs
};

template <typename TX, typename TY, int V, int K>
__global__ void __launch_bounds__(kThr) gn_row_forward_kernel(const GnArgs a, int team) {
    const int cg = a.C / a.G;
    const int lane = threadIdx.x & (team - 1);
    const long long teams = static_cast<long long>(gridDim.x) * (kThr / team);
    const long long me = static_cast<long long>(blockIdx.x) * (kThr / team) + threadIdx.x / team;
    const TX *x = static_cast<const TX *>(a.x), *gate = static_cast<const TX *>(a.gate);
    TY *y = static_cast<TY *>(a.y);
    const long long all = static_cast<long long>(a.N) * a.G;
    const long long trips = (all + teams - 1) / teams;
    const float inv = 1.f / cg;
    for (long long i = 0; i < trips; ++i) {
        const long long slab = i * teams + me;
        const bool on = slab < all;
        const long long n = on ? slab / a.G : 0;
        const int g = on ? static_cast<int>(slab % a.G) : 0;
        const bool live = on && (a.lengths == nullptr || a.lengths[n] > 0);
        const long long base = n * a.C + static_cast<long long>(g) * cg;
        float v[K][V];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * team + lane) * V;
            if (live && c < cg) {
                load<V>(x + base + c, v[k]);
            } else {
#pragma unroll
                for (int u = 0; u < V; ++u) v[k][u] = 0.f;
            }
#pragma unroll
            for (int u = 0; u < V; ++u) sum += v[k][u];
        }
        for (int m = team >> 1; m > 0; m >>= 1) sum += __shfl_xor_sync(~0u, sum, m);
        const float mean = sum * inv;
        float m2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if ((k * team + lane) * V < cg) {
#pragma unroll
                for (int u = 0; u < V; ++u) m2 = fmaf(v[k][u] - mean, v[k][u] - mean, m2);
            }
        for (int m = team >> 1; m > 0; m >>= 1) m2 += __shfl_xor_sync(~0u, m2, m);
        const float rstd = rsqrtf(fmaf(live ? m2 : 0.f, inv, a.eps));
        if (on && lane == 0) *reinterpret_cast<float2 *>(a.stats + slab * 2) = make_float2(mean, rstd);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * team + lane) * V;
            if (!on || c >= cg) continue;
            float o[V] = {};
            if (live) {
                float w[V], b[V], q[V];
                load_wb<V>(a, g * cg + c, w, b);
                if (gate != nullptr) load<V>(gate + base + c, q);
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    const float z = fmaf((v[k][u] - mean) * rstd, w[u], b[u]);
                    o[u] = gate != nullptr ? z * act_of(q[u], a.act) : act_of(z, a.act);
                }
            }
            store<V>(y + base + c, o);
        }
    }
}

// Backward: CTA (bx, by) takes the groups of column block by and the rows bx, bx + gridDim.x, ... ; its sums of
// dw and db over those rows go to part[bx][2][C].
template <typename TX, typename TY, int V, int K>
__global__ void __launch_bounds__(kThr) gn_row_backward_kernel(const GnArgs a, int team, float *part) {
    extern __shared__ float red[];  // [rows in flight][dw, db][this CTA's channels]
    const int cg = a.C / a.G;
    const int per = kThr / team;                      // teams per CTA
    const int gpc = min(per, a.G);                    // groups per CTA
    const int rows = per / gpc;                       // rows in flight
    const int tm = threadIdx.x / team, lane = threadIdx.x & (team - 1);
    const int g = blockIdx.y * gpc + tm % gpc, rr = tm / gpc;
    const bool have = g < a.G && rr < rows;
    const TX *x = static_cast<const TX *>(a.x), *gate = static_cast<const TX *>(a.gate);
    const TY *dy = static_cast<const TY *>(a.y);
    TX *dx = static_cast<TX *>(a.dx), *dgate = static_cast<TX *>(a.dgate);
    const float inv = 1.f / cg;
    float w[K][V], b[K][V], dw[K][V], db[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * team + lane) * V;
#pragma unroll
        for (int u = 0; u < V; ++u) w[k][u] = 1.f, b[k][u] = dw[k][u] = db[k][u] = 0.f;
        if (have && c < cg) load_wb<V>(a, g * cg + c, w[k], b[k]);
    }
    const long long step = static_cast<long long>(gridDim.x) * rows;
    for (long long n0 = static_cast<long long>(blockIdx.x) * rows; n0 < a.N; n0 += step) {
        const long long n = n0 + rr;
        const bool on = have && n < a.N;
        const bool live = on && (a.lengths == nullptr || a.lengths[n] > 0);
        const long long base = n * a.C + static_cast<long long>(g) * cg;
        float mean = 0.f, rstd = 0.f;
        if (live) {
            const float2 st = *reinterpret_cast<const float2 *>(a.stats + (static_cast<long long>(n) * a.G + g) * 2);
            mean = st.x, rstd = st.y;
        }
        float xh[K][V], dh[K][V];  // xhat, w dz
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * team + lane) * V;
            const bool in = live && c < cg;
            float t[V];
#pragma unroll
            for (int u = 0; u < V; ++u) xh[k][u] = dh[k][u] = t[u] = 0.f;
            if (in) {
                load<V>(x + base + c, xh[k]);
                load<V>(dy + base + c, t);
            }
            if (gate != nullptr) {
                float q[V] = {}, dg[V];
                if (in) load<V>(gate + base + c, q);
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    xh[k][u] = (xh[k][u] - mean) * rstd;
                    const float z = fmaf(xh[k][u], w[k][u], b[k][u]);
                    dg[u] = t[u] * z * act_slope(q[u], a.act);
                    t[u] *= act_of(q[u], a.act);
                }
                if (on && c < cg) {
                    if (!live) {
#pragma unroll
                        for (int u = 0; u < V; ++u) dg[u] = 0.f;
                    }
                    store<V>(dgate + base + c, dg);
                }
            } else {
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    xh[k][u] = (xh[k][u] - mean) * rstd;
                    t[u] *= act_slope(fmaf(xh[k][u], w[k][u], b[k][u]), a.act);
                }
            }
            if (in) {
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    db[k][u] += t[u];
                    dw[k][u] = fmaf(t[u], xh[k][u], dw[k][u]);
                    dh[k][u] = t[u] * w[k][u];
                    s1 += dh[k][u];
                    s2 = fmaf(dh[k][u], xh[k][u], s2);
                }
            }
        }
        for (int m = team >> 1; m > 0; m >>= 1) {
            s1 += __shfl_xor_sync(~0u, s1, m);
            s2 += __shfl_xor_sync(~0u, s2, m);
        }
        s1 *= inv;
        s2 *= inv;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * team + lane) * V;
            if (!on || c >= cg) continue;
            float o[V] = {};
            if (live) {
#pragma unroll
                for (int u = 0; u < V; ++u) o[u] = rstd * (dh[k][u] - s1 - xh[k][u] * s2);
            }
            store<V>(dx + base + c, o);
        }
    }
    // rows in flight summed in order, then this CTA's partial sums out
    const int width = gpc * cg;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * team + lane) * V;
        if (rr < rows && c < cg) {
#pragma unroll
            for (int u = 0; u < V; ++u) {
                red[(rr * 2 + 0) * width + (tm % gpc) * cg + c + u] = dw[k][u];
                red[(rr * 2 + 1) * width + (tm % gpc) * cg + c + u] = db[k][u];
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * width; i += kThr) {
        const int which = i / width, c = i % width, ch = blockIdx.y * width + c;
        if (ch >= a.C) continue;
        float s = 0.f;
        for (int q = 0; q < rows; ++q) s += red[(q * 2 + which) * width + c];
        part[(static_cast<long long>(blockIdx.x) * 2 + which) * a.C + ch] = s;
    }
}

// dw, db [C] = sums of part [rows][2][C] in row order: 8 row slices per CTA of 32 channels, then across them
__global__ void __launch_bounds__(256) gn_param_sum_kernel(const float *part, int rows, int C, float *dw, float *db) {
    __shared__ float red[8][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), sl = threadIdx.x >> 5, which = blockIdx.y;
    float s = 0.f;
    if (c < C)
        for (int r = sl; r < rows; r += 8) s += part[(static_cast<long long>(r) * 2 + which) * C + c];
    red[sl][threadIdx.x & 31] = s;
    __syncthreads();
    if (sl == 0 && c < C) {
        for (int q = 1; q < 8; ++q) s += red[q][threadIdx.x];
        float *out = which == 0 ? dw : db;
        if (out != nullptr) out[c] = s;
    }
}

// ---- statistics over a sequence ------------------------------------------------------------------------------

// A CTA takes `rows` rows of one n.  Its threads span the channels (vectors of V within one group) and, where
// there are fewer vectors than threads, several rows at once.
struct Span {
    int cols, par;  // vectors per row; rows in flight
};
template <int V>
__device__ __forceinline__ Span span_of(const GnArgs &a) {
    const int cols = a.C / V;
    return {cols, cols >= kThr ? 1 : kThr / cols};
}

// part[n][chunk][g] = moments of group g in this CTA's rows
template <typename TX, int V>
__global__ void __launch_bounds__(kThr) gn_stats_kernel(const GnArgs a, int rows, int chunks, Moments *part) {
    constexpr int RB = 32 / V < 8 ? 32 / V : 8;  // rows a thread holds at a time
    __shared__ Moments red[kThr];
    extern __shared__ Moments acc[];  // [G]
    const int n = static_cast<int>(blockIdx.x / chunks), ch = static_cast<int>(blockIdx.x % chunks), L = row_count(a, n);
    const int lo = static_cast<int>(min(static_cast<long long>(ch) * rows, static_cast<long long>(L)));
    const int hi = static_cast<int>(min((ch + 1ll) * rows, static_cast<long long>(L)));
    const TX *x = static_cast<const TX *>(a.x) + static_cast<long long>(n) * a.S * a.C;
    const Span sp = span_of<V>(a);
    const int cg = a.C / a.G, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int g = threadIdx.x; g < a.G; g += kThr) acc[g] = {0.f, 0.f, 0.f};
    for (int cb = 0; cb < sp.cols; cb += kThr) {
        const int width = min(kThr, sp.cols - cb);
        const int r0 = sp.par == 1 ? 0 : threadIdx.x / sp.cols;
        const int col = sp.par == 1 ? threadIdx.x : threadIdx.x % sp.cols;
        Moments m = {0.f, 0.f, 0.f};
        if (col < width && r0 < sp.par) {
            const TX *p = x + static_cast<long long>(cb + col) * V;
            for (int s = lo + r0; s < hi; s += RB * sp.par) {
                float v[RB][V];
                int cnt = 0;
                float sum = 0.f;
#pragma unroll
                for (int u = 0; u < RB; ++u)
                    if (s + u * sp.par < hi) {
                        load<V>(p + static_cast<long long>(s + u * sp.par) * a.C, v[u]);
                        ++cnt;
                    } else {
#pragma unroll
                        for (int i = 0; i < V; ++i) v[u][i] = 0.f;
                    }
#pragma unroll
                for (int u = 0; u < RB; ++u)
#pragma unroll
                    for (int i = 0; i < V; ++i) sum += v[u][i];
                const float nb = static_cast<float>(cnt * V), mb = sum / nb;
                float m2 = 0.f;
#pragma unroll
                for (int u = 0; u < RB; ++u)
                    if (u < cnt) {
#pragma unroll
                        for (int i = 0; i < V; ++i) m2 = fmaf(v[u][i] - mb, v[u][i] - mb, m2);
                    }
                m = join(m, {nb, mb, m2});
            }
        }
        __syncthreads();
        red[threadIdx.x] = m;
        __syncthreads();
        // the groups of this column block, a warp each: its vectors times the rows in flight
        const int g_lo = cb * V / cg, g_hi = (min(sp.cols, cb + width) * V - 1) / cg;
        for (int g = g_lo + warp; g <= g_hi; g += kThr / 32) {
            const int c_lo = max(g * cg / V, cb) - cb, c_hi = min((g + 1) * cg / V, cb + width) - cb;
            const int w = c_hi - c_lo;
            Moments t = {0.f, 0.f, 0.f};
            for (int i = lane; i < w * sp.par; i += 32) t = join(t, red[(i / w) * (sp.par == 1 ? 0 : sp.cols) + c_lo + i % w]);
#pragma unroll
            for (int q = 16; q > 0; q >>= 1) t = join(t, shuffle_xor(t, q));
            if (lane == 0) acc[g] = join(acc[g], t);
        }
    }
    __syncthreads();
    Moments *out = part + static_cast<long long>(blockIdx.x) * a.G;
    for (int g = threadIdx.x; g < a.G; g += kThr) out[g] = acc[g];
}

__global__ void __launch_bounds__(kThr) gn_stats_join_kernel(const GnArgs a, int chunks, const Moments *part) {
    const long long i = (static_cast<long long>(blockIdx.x) * kThr + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (i >= static_cast<long long>(a.N) * a.G) return;
    const long long n = i / a.G, g = i % a.G;
    Moments t = {0.f, 0.f, 0.f};
    for (int q = lane; q < chunks; q += 32) t = join(t, part[(n * chunks + q) * a.G + g]);
#pragma unroll
    for (int q = 16; q > 0; q >>= 1) t = join(t, shuffle_xor(t, q));
    if (lane == 0) {
        const float var = t.n > 0.f ? t.m2 / t.n : 0.f;
        *reinterpret_cast<float2 *>(a.stats + i * 2) = make_float2(t.mean, rsqrtf(var + a.eps));
    }
}

template <typename TX, typename TY, int V>
__global__ void __launch_bounds__(kThr) gn_apply_kernel(const GnArgs a, int rows, int chunks) {
    const int n = static_cast<int>(blockIdx.x / chunks), ch = static_cast<int>(blockIdx.x % chunks), L = row_count(a, n);
    const long long lo = static_cast<long long>(ch) * rows;
    const int hi = static_cast<int>(min(lo + rows, static_cast<long long>(a.S)));
    const long long nb = static_cast<long long>(n) * a.S * a.C;
    const TX *x = static_cast<const TX *>(a.x) + nb;
    const TX *gate = a.gate == nullptr ? nullptr : static_cast<const TX *>(a.gate) + nb;
    TY *y = static_cast<TY *>(a.y) + nb;
    const Span sp = span_of<V>(a);
    const int r0 = sp.par == 1 ? 0 : threadIdx.x / sp.cols;
    if (r0 >= sp.par) return;
    for (int col = sp.par == 1 ? threadIdx.x : threadIdx.x % sp.cols; col < sp.cols; col += sp.par == 1 ? kThr : sp.cols) {
        const int c = col * V, g = c / (a.C / a.G);
        const float2 st = *reinterpret_cast<const float2 *>(a.stats + (static_cast<long long>(n) * a.G + g) * 2);
        float w[V], b[V];
        load_wb<V>(a, c, w, b);
#pragma unroll
        for (int i = 0; i < V; ++i) {  // z = x * w' + b'' after the mean is taken off
            w[i] *= st.y;
        }
#pragma unroll 4
        for (int s = static_cast<int>(lo) + r0; s < hi; s += sp.par) {
            const long long at = static_cast<long long>(s) * a.C + c;
            float o[V] = {};
            if (s < L) {
                float v[V], q[V];
                load<V>(x + at, v);
                if (gate != nullptr) load<V>(gate + at, q);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float z = fmaf(v[i] - st.x, w[i], b[i]);
                    o[i] = gate != nullptr ? z * act_of(q[i], a.act) : act_of(z, a.act);
                }
            }
            store<V>(y + at, o);
        }
    }
}

// dz of one element, and xhat; with a gate also dgate
template <bool GATE>
__device__ __forceinline__ float dz_of(const GnArgs &a, float dy, float xhat, float w, float b, float q, float *dg) {
    const float z = fmaf(xhat, w, b);
    if (GATE) {
        if (dg != nullptr) *dg = dy * z * act_slope(q, a.act);
        return dy * act_of(q, a.act);
    }
    return dy * act_slope(z, a.act);
}

// part[n][chunk][2][C]: sums of dz xhat and of dz over this CTA's rows
template <typename TX, typename TY, int V, bool GATE>
__global__ void __launch_bounds__(kThr) gn_channel_sum_kernel(const GnArgs a, int rows, int chunks, float *part) {
    __shared__ float red[2][kThr * V];
    const int n = static_cast<int>(blockIdx.x / chunks), ch = static_cast<int>(blockIdx.x % chunks), L = row_count(a, n);
    const long long lo = static_cast<long long>(ch) * rows;
    const int hi = static_cast<int>(min(lo + rows, static_cast<long long>(L)));
    const long long nb = static_cast<long long>(n) * a.S * a.C;
    const TX *x = static_cast<const TX *>(a.x) + nb, *gate = GATE ? static_cast<const TX *>(a.gate) + nb : nullptr;
    const TY *dy = static_cast<const TY *>(a.y) + nb;
    const Span sp = span_of<V>(a);
    float *out = part + static_cast<long long>(blockIdx.x) * 2 * a.C;
    for (int cb = 0; cb < sp.cols; cb += kThr) {
        const int width = min(kThr, sp.cols - cb);
        const int r0 = sp.par == 1 ? 0 : threadIdx.x / sp.cols;
        const int col = sp.par == 1 ? threadIdx.x : threadIdx.x % sp.cols;
        float dw[V] = {}, db[V] = {};
        if (col < width && r0 < sp.par) {
            const int c = (cb + col) * V, g = c / (a.C / a.G);
            const float2 st = *reinterpret_cast<const float2 *>(a.stats + (static_cast<long long>(n) * a.G + g) * 2);
            float w[V], b[V];
            load_wb<V>(a, c, w, b);
#pragma unroll 4
            for (long long s = lo + r0; s < hi; s += sp.par) {
                float v[V], t[V], q[V] = {};
                load<V>(x + s * a.C + c, v);
                load<V>(dy + s * a.C + c, t);
                if (GATE) load<V>(gate + s * a.C + c, q);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xh = (v[i] - st.x) * st.y;
                    const float dz = dz_of<GATE>(a, t[i], xh, w[i], b[i], q[i], nullptr);
                    db[i] += dz;
                    dw[i] = fmaf(dz, xh, dw[i]);
                }
            }
        }
        if (sp.par == 1) {
            if (col < width) {
                store<V>(out + (cb + col) * V, dw);
                store<V>(out + a.C + (cb + col) * V, db);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) red[0][threadIdx.x * V + i] = dw[i], red[1][threadIdx.x * V + i] = db[i];
            __syncthreads();
            for (int i = threadIdx.x; i < 2 * a.C; i += kThr) {
                const int which = i / a.C, c = i % a.C;
                float s = 0.f;
                for (int q = 0; q < sp.par; ++q) s += red[which][q * a.C + c];
                out[i] = s;
            }
        }
    }
}

// One CTA per n: channel sums over the chunks -> chan[n][2][C], group sums of w dz and w dz xhat -> gsum[n][g][2]
__global__ void __launch_bounds__(kThr) gn_channel_join_kernel(const GnArgs a, int chunks, const float *part,
                                                               float *chan, float *gsum) {
    const int n = blockIdx.x;
    const float *p = part + static_cast<long long>(n) * chunks * 2 * a.C;
    float *ch = chan + static_cast<long long>(n) * 2 * a.C;
    for (int i = threadIdx.x; i < 2 * a.C; i += kThr) {
        float s = 0.f;
#pragma unroll 8
        for (int q = 0; q < chunks; ++q) s += p[static_cast<long long>(q) * 2 * a.C + i];
        ch[i] = s;
    }
    __syncthreads();
    const int cg = a.C / a.G, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int g = warp; g < a.G; g += kThr / 32) {
        float s1 = 0.f, s2 = 0.f;
        for (int c = g * cg + lane; c < (g + 1) * cg; c += 32) {
            const float w = a.weight != nullptr ? a.weight[c] : 1.f;
            s2 = fmaf(w, ch[c], s2);
            s1 = fmaf(w, ch[a.C + c], s1);
        }
#pragma unroll
        for (int q = 16; q > 0; q >>= 1) s1 += __shfl_xor_sync(~0u, s1, q), s2 += __shfl_xor_sync(~0u, s2, q);
        if (lane == 0) *reinterpret_cast<float2 *>(gsum + (static_cast<long long>(n) * a.G + g) * 2) = make_float2(s1, s2);
    }
}

template <typename TX, typename TY, int V, bool GATE>
__global__ void __launch_bounds__(kThr) gn_backward_apply_kernel(const GnArgs a, int rows, int chunks, const float *gsum) {
    const int n = static_cast<int>(blockIdx.x / chunks), ch = static_cast<int>(blockIdx.x % chunks), L = row_count(a, n);
    const long long lo = static_cast<long long>(ch) * rows;
    const long long hi = min(lo + rows, static_cast<long long>(a.S));
    const long long nb = static_cast<long long>(n) * a.S * a.C;
    const TX *x = static_cast<const TX *>(a.x) + nb, *gate = GATE ? static_cast<const TX *>(a.gate) + nb : nullptr;
    const TY *dy = static_cast<const TY *>(a.y) + nb;
    TX *dx = static_cast<TX *>(a.dx) + nb, *dgate = GATE ? static_cast<TX *>(a.dgate) + nb : nullptr;
    const Span sp = span_of<V>(a);
    const int r0 = sp.par == 1 ? 0 : threadIdx.x / sp.cols;
    if (r0 >= sp.par) return;
    const int cg = a.C / a.G;
    const float inv = 1.f / (static_cast<float>(max(L, 1)) * cg);
    for (int col = sp.par == 1 ? threadIdx.x : threadIdx.x % sp.cols; col < sp.cols; col += sp.par == 1 ? kThr : sp.cols) {
        const int c = col * V, g = c / cg;
        const long long sg = (static_cast<long long>(n) * a.G + g) * 2;
        const float2 st = *reinterpret_cast<const float2 *>(a.stats + sg);
        float2 gs = *reinterpret_cast<const float2 *>(gsum + sg);
        gs.x *= inv, gs.y *= inv;
        float w[V], b[V];
        load_wb<V>(a, c, w, b);
#pragma unroll 2
        for (long long s = lo + r0; s < hi; s += sp.par) {
            const long long at = s * a.C + c;
            float o[V] = {}, dg[V] = {};
            if (s < L) {
                float v[V], t[V], q[V] = {};
                load<V>(x + at, v);
                load<V>(dy + at, t);
                if (GATE) load<V>(gate + at, q);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xh = (v[i] - st.x) * st.y;
                    const float dz = dz_of<GATE>(a, t[i], xh, w[i], b[i], q[i], &dg[i]);
                    o[i] = st.y * (w[i] * dz - gs.x - xh * gs.y);
                }
            }
            store<V>(dx + at, o);
            if (GATE) store<V>(dgate + at, dg);
        }
    }
}

// ---- plans and dispatch --------------------------------------------------------------------------------------

constexpr int kRowMost = 1024;  // channels of a group that a warp holds in registers (32 per lane)

bool row_regime(const GnArgs &a) { return a.S == 1 && a.C / a.G <= kRowMost; }
int vec_of(const GnArgs &a) {
    const int cg = a.C / a.G;
    return cg % 8 == 0 ? 8 : cg % 4 == 0 ? 4 : 1;
}
int team_of(const GnArgs &a, int V) {
    const int need = (a.C / a.G + V - 1) / V;
    int t = 1;
    while (t < need && t < 32) t *= 2;
    return t;
}
// rows per CTA: 8 CTAs of 256 threads per SM, at least about 16K elements each
int chunk_rows(const GnArgs &a) {
    const long long all = static_cast<long long>(a.N) * a.S;
    long long rows = (all + 148 * 8 - 1) / (148 * 8);
    const long long least = (16384 + a.C - 1) / a.C;
    if (rows < least) rows = least;
    if (rows > a.S) rows = a.S;
    return static_cast<int>(rows);
}
int row_backward_ctas(const GnArgs &a, int V) {
    const int per = kThr / team_of(a, V), gpc = per < a.G ? per : a.G, rows = per / gpc;
    const int by = (a.G + gpc - 1) / gpc;
    long long bx = (148 * 4 + by - 1) / by;
    const long long most = (a.N + rows - 1) / rows;
    if (bx > most) bx = most;
    return static_cast<int>(bx < 1 ? 1 : bx);
}
size_t al(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <typename TX, typename TY, int V, int K>
cudaError_t row_forward(const GnArgs &a, cudaStream_t s) {
    const int team = team_of(a, V);
    const long long ctas = (static_cast<long long>(a.N) * a.G * team + kThr - 1) / kThr;
    const unsigned grid = static_cast<unsigned>(ctas < 148 * 16 ? ctas : 148 * 16);
    gn_row_forward_kernel<TX, TY, V, K><<<grid, kThr, 0, s>>>(a, team);
    return cudaGetLastError();
}

template <typename TX, typename TY, int V, int K>
cudaError_t row_backward(const GnArgs &a, cudaStream_t s) {
    const int team = team_of(a, V), per = kThr / team, gpc = per < a.G ? per : a.G, rows = per / gpc;
    const int bx = row_backward_ctas(a, V);
    const dim3 grid(bx, (a.G + gpc - 1) / gpc);
    const int smem = rows * 2 * gpc * (a.C / a.G) * 4;
    auto k = gn_row_backward_kernel<TX, TY, V, K>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    k<<<grid, kThr, smem, s>>>(a, team, reinterpret_cast<float *>(a.ws));
    gn_param_sum_kernel<<<dim3((a.C + 31) / 32, 2), 256, 0, s>>>(reinterpret_cast<float *>(a.ws), bx, a.C, a.dweight,
                                                                a.dbias);
    return cudaGetLastError();
}

template <typename TX, typename TY, int V>
cudaError_t seq_forward(const GnArgs &a, cudaStream_t s) {
    const int rows = chunk_rows(a), chunks = (a.S + rows - 1) / rows;
    Moments *part = reinterpret_cast<Moments *>(a.ws);
    const unsigned grid = static_cast<unsigned>(chunks) * a.N;
    gn_stats_kernel<TX, V><<<grid, kThr, a.G * sizeof(Moments), s>>>(a, rows, chunks, part);
    const long long warps = static_cast<long long>(a.N) * a.G;
    gn_stats_join_kernel<<<static_cast<unsigned>((warps * 32 + kThr - 1) / kThr), kThr, 0, s>>>(a, chunks, part);
    gn_apply_kernel<TX, TY, V><<<grid, kThr, 0, s>>>(a, rows, chunks);
    return cudaGetLastError();
}

template <typename TX, typename TY, int V, bool GATE>
cudaError_t seq_backward_g(const GnArgs &a, cudaStream_t s) {
    const int rows = chunk_rows(a), chunks = (a.S + rows - 1) / rows;
    const unsigned grid = static_cast<unsigned>(chunks) * a.N;
    float *part = reinterpret_cast<float *>(a.ws);
    float *chan = reinterpret_cast<float *>(a.ws + al(static_cast<size_t>(a.N) * chunks * 2 * a.C * 4));
    float *gsum = reinterpret_cast<float *>(reinterpret_cast<char *>(chan) + al(static_cast<size_t>(a.N) * 2 * a.C * 4));
    gn_channel_sum_kernel<TX, TY, V, GATE><<<grid, kThr, 0, s>>>(a, rows, chunks, part);
    gn_channel_join_kernel<<<a.N, kThr, 0, s>>>(a, chunks, part, chan, gsum);
    gn_backward_apply_kernel<TX, TY, V, GATE><<<grid, kThr, 0, s>>>(a, rows, chunks, gsum);
    gn_param_sum_kernel<<<dim3((a.C + 31) / 32, 2), 256, 0, s>>>(chan, a.N, a.C, a.dweight, a.dbias);
    return cudaGetLastError();
}

template <typename TX, typename TY, bool BACK>
cudaError_t dispatch(const GnArgs &a, cudaStream_t s) {
    const int V = vec_of(a);
    if (row_regime(a)) {
        const int k = (a.C / a.G + 32 * V - 1) / (32 * V);  // vectors per lane of a full warp
        if (BACK) {
            if (V == 8) return k <= 1 ? row_backward<TX, TY, 8, 1>(a, s) : row_backward<TX, TY, 8, 4>(a, s);
            if (V == 4) return k <= 1 ? row_backward<TX, TY, 4, 1>(a, s) : row_backward<TX, TY, 4, 8>(a, s);
            return k <= 4 ? row_backward<TX, TY, 1, 4>(a, s) : row_backward<TX, TY, 1, 32>(a, s);
        }
        if (V == 8) return k <= 1 ? row_forward<TX, TY, 8, 1>(a, s) : row_forward<TX, TY, 8, 4>(a, s);
        if (V == 4) return k <= 1 ? row_forward<TX, TY, 4, 1>(a, s) : row_forward<TX, TY, 4, 8>(a, s);
        return k <= 4 ? row_forward<TX, TY, 1, 4>(a, s) : row_forward<TX, TY, 1, 32>(a, s);
    }
    if (BACK) {
        if (a.gate != nullptr)
            return V == 8   ? seq_backward_g<TX, TY, 8, true>(a, s)
                   : V == 4 ? seq_backward_g<TX, TY, 4, true>(a, s)
                            : seq_backward_g<TX, TY, 1, true>(a, s);
        return V == 8   ? seq_backward_g<TX, TY, 8, false>(a, s)
               : V == 4 ? seq_backward_g<TX, TY, 4, false>(a, s)
                        : seq_backward_g<TX, TY, 1, false>(a, s);
    }
    return V == 8 ? seq_forward<TX, TY, 8>(a, s) : V == 4 ? seq_forward<TX, TY, 4>(a, s) : seq_forward<TX, TY, 1>(a, s);
}

template <bool BACK>
cudaError_t by_type(const GnArgs &a, cudaStream_t s) {
    if (a.x_dtype == PARARNN_F32)
        return a.y_dtype == PARARNN_F32 ? dispatch<float, float, BACK>(a, s) : dispatch<float, __nv_bfloat16, BACK>(a, s);
    return a.y_dtype == PARARNN_F32 ? dispatch<__nv_bfloat16, float, BACK>(a, s)
                                    : dispatch<__nv_bfloat16, __nv_bfloat16, BACK>(a, s);
}

}  // namespace

size_t gn_ws_bytes(const GnArgs &a, bool backward) {
    if (row_regime(a))
        return backward ? al(static_cast<size_t>(row_backward_ctas(a, vec_of(a))) * 2 * a.C * 4) : 256;
    const int rows = chunk_rows(a), chunks = (a.S + rows - 1) / rows;
    if (!backward) return al(static_cast<size_t>(a.N) * chunks * a.G * sizeof(Moments));
    return al(static_cast<size_t>(a.N) * chunks * 2 * a.C * 4) + al(static_cast<size_t>(a.N) * 2 * a.C * 4) +
           al(static_cast<size_t>(a.N) * a.G * 8);
}

cudaError_t launch_gn_forward(const GnArgs &a, cudaStream_t s) { return by_type<false>(a, s); }
cudaError_t launch_gn_backward(const GnArgs &a, cudaStream_t s) { return by_type<true>(a, s); }

}  // namespace pararnn
