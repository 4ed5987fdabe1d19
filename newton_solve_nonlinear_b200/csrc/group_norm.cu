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
//
// Measured: 32768 rows of 16 heads of 128, bf16 under a gate, 92 us, 0.67 of a copy of its bytes.  It waits for loads: 128
// registers a thread leave a quarter of the warps (24 %), and these issue in 54 % of the cycles, about 30 instructions per
// element, most of them unpacking and the sigmoid; loading the next rows during a row's arithmetic gave 106 us, since
// registers run out.  Its backward pass on 8192 rows 60 us, 0.43, of which the sum of the CTAs' partial rows takes 5.
// [16, 65536, 64] fp32 to bf16 126 us: 57 for the statistics and 69 to read x again and write y, 0.72 and 0.89 of a copy's
// rate, as they follow one another in a call (47 and 80 alone under a profiler, from cold caches); registers limit the
// warps in flight.  Ragged [8, 1000, 640] backward 43 us, three launches that wait for one another (16, 6 and 17).
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

// d = a * b + c on V elements, two at a time (fma.rn.f32x2 is two fp32 FMAs in one instruction: these kernels are
// bound by instructions before they are bound by memory)
__device__ __forceinline__ void fma_pair(float &d0, float &d1, float a0, float a1, float b0, float b1, float c0, float c1) {
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mul_pair(float &d0, float &d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void add_pair(float &d0, float &d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
template <int V>
__device__ __forceinline__ void vfma(float (&d)[V], const float (&a)[V], const float (&b)[V], const float (&c)[V]) {
    if constexpr (V == 1) d[0] = fmaf(a[0], b[0], c[0]);
    else
#pragma unroll
        for (int i = 0; i < V; i += 2) fma_pair(d[i], d[i + 1], a[i], a[i + 1], b[i], b[i + 1], c[i], c[i + 1]);
}
template <int V>
__device__ __forceinline__ void vmul(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
    if constexpr (V == 1) d[0] = a[0] * b[0];
    else
#pragma unroll
        for (int i = 0; i < V; i += 2) mul_pair(d[i], d[i + 1], a[i], a[i + 1], b[i], b[i + 1]);
}
template <int V>
__device__ __forceinline__ void vscale(float (&d)[V], const float (&a)[V], float s) {
    if constexpr (V == 1) d[0] = a[0] * s;
    else
#pragma unroll
        for (int i = 0; i < V; i += 2) mul_pair(d[i], d[i + 1], a[i], a[i + 1], s, s);
}
template <int V>
__device__ __forceinline__ void vshift(float (&d)[V], const float (&a)[V], float s) {
    if constexpr (V == 1) d[0] = a[0] + s;
    else
#pragma unroll
        for (int i = 0; i < V; i += 2) add_pair(d[i], d[i + 1], a[i], a[i + 1], s, s);
}
template <int V>
__device__ __forceinline__ void vadd(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
    if constexpr (V == 1) d[0] = a[0] + b[0];
    else
#pragma unroll
        for (int i = 0; i < V; i += 2) add_pair(d[i], d[i + 1], a[i], a[i + 1], b[i], b[i + 1]);
}
// sum of V elements, sum of a b
template <int V>
__device__ __forceinline__ float vsum(const float (&a)[V]) {
    if constexpr (V == 1) return a[0];
    float s0 = a[0], s1 = a[V > 1 ? 1 : 0];
#pragma unroll
    for (int i = 2; i < V; i += 2) add_pair(s0, s1, s0, s1, a[i], a[i + 1]);
    return s0 + s1;
}
template <int V>
__device__ __forceinline__ float vdot(const float (&a)[V], const float (&b)[V]) {
    if constexpr (V == 1) return a[0] * b[0];
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < V; i += 2) fma_pair(s0, s1, a[i], a[i + 1], b[i], b[i + 1], s0, s1);
    return s0 + s1;
}

// 1 / (1 + exp(-z)), by the fast exponential, which is documented as within 2 + floor(|1.173 z|) ulp, and the approximate
// reciprocal, within one: the result is within (1 - s)(2 + 1.173 |z|) + 1.5 ulp, so within 3 where z > 0, and, as the
// exponential's argument is large, more relative to a small result where z is far below zero (15 at -10, 97 at -80).
// GELU's slope takes the same exponential of -z^2 / 2.
__device__ __forceinline__ float sigmoid(float z) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + __expf(-z)));
    return r;
}
// z = act(z) for V elements, and with it s = act'(z); one branch on the kind for all of them
template <int V>
__device__ __forceinline__ void act_of(float (&z)[V], int act) {
    if (act == PARARNN_ACT_SILU) {
        float s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = sigmoid(z[i]);
        vmul<V>(z, z, s);
    } else if (act == PARARNN_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] *= normcdff(z[i]);
    }
}
template <int V>
__device__ __forceinline__ void act_and_slope(float (&z)[V], float (&s)[V], int act) {
    if (act == PARARNN_ACT_SILU) {  // a = z g, act' = g + a (1 - g) = (g + a) - a g
        float g[V], h[V];
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = sigmoid(z[i]);
        vmul<V>(z, z, g);
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] = 1.f - g[i];
        vfma<V>(s, z, h, g);
    } else if (act == PARARNN_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float p = normcdff(z[i]);
            s[i] = fmaf(z[i] * 0.3989422804014327f, __expf(-0.5f * z[i] * z[i]), p);
            z[i] *= p;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = 1.f;
    }
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

// A team of `team` lanes (a power of two) holds K vectors of V channels per lane of one group: channels
// (k team + lane) V + i.  A CTA covers `gpc` groups and `rows` rows at a time (blockIdx.y: which groups), so a team
// keeps its group and its weights stay in registers.  R rows are loaded before the first is used.
struct Teams {
    int team, gpc, rows;
};
__device__ __forceinline__ Teams teams_of(int G, int team) {
    const int per = kThr / team, gpc = min(per, G);
    return {team, gpc, per / gpc};
}

template <typename T, int V>
struct Raw {  // V elements as they come from memory
    static constexpr int WORDS = sizeof(T) * V / 4 < 1 ? 1 : sizeof(T) * V / 4;
    unsigned u[WORDS];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) u[i] = 0u;
    }
    __device__ __forceinline__ void get(const T *p) {
        if constexpr (sizeof(T) * V == 2) {
            u[0] = *reinterpret_cast<const unsigned short *>(p);
        } else if constexpr (sizeof(T) * V == 4) {
            u[0] = *reinterpret_cast<const unsigned *>(p);
        } else if constexpr (sizeof(T) * V == 8) {
            const uint2 x = *reinterpret_cast<const uint2 *>(p);
            u[0] = x.x, u[1] = x.y;
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; i += 4) {
                const uint4 x = *reinterpret_cast<const uint4 *>(reinterpret_cast<const unsigned *>(p) + i);
                u[i] = x.x, u[i + 1] = x.y, u[i + 2] = x.z, u[i + 3] = x.w;
            }
        }
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(u[i]);
        else return (i & 1) ? __uint_as_float(u[i >> 1] & 0xffff0000u) : __uint_as_float(u[i >> 1] << 16);
    }
};

template <typename TX, typename TY, int V, int K, int R>
__global__ void __launch_bounds__(kThr, V * K <= 16 ? 2 : 1) gn_row_forward_kernel(const GnArgs a, int team) {
    const int cg = a.C / a.G;
    const Teams tt = teams_of(a.G, team);
    const int tm = threadIdx.x / team, lane = threadIdx.x & (team - 1);
    const int g = blockIdx.y * tt.gpc + tm % tt.gpc, rr = tm / tt.gpc;
    const bool have = g < a.G && rr < tt.rows;
    const TX *x = static_cast<const TX *>(a.x), *gate = static_cast<const TX *>(a.gate);
    TY *y = static_cast<TY *>(a.y);
    const float inv = 1.f / cg;
    float w[K][V], b[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * team + lane) * V;
#pragma unroll
        for (int u = 0; u < V; ++u) w[k][u] = 1.f, b[k][u] = 0.f;
        if (have && c < cg) load_wb<V>(a, g * cg + c, w[k], b[k]);
    }
    const long long step = static_cast<long long>(gridDim.x) * tt.rows;
    for (long long n0 = static_cast<long long>(blockIdx.x) * tt.rows + rr; n0 - rr < a.N; n0 += step * R) {
        Raw<TX, V> v[R][K], q[R][K];
        bool on[R], live[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const long long n = n0 + r * step;
            on[r] = have && n < a.N;
            live[r] = on[r] && (a.lengths == nullptr || a.lengths[n] > 0);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * team + lane) * V;
                v[r][k].zero();
                q[r][k].zero();
                if (live[r] && c < cg) {
                    const long long at = n * a.C + static_cast<long long>(g) * cg + c;
                    v[r][k].get(x + at);
                    if (gate != nullptr) q[r][k].get(gate + at);
                }
            }
        }
        float mean[R], m2[R], d[R][K][V];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int u = 0; u < V; ++u) d[r][k][u] = v[r][k].at(u);
                mean[r] += vsum<V>(d[r][k]);
            }
        }
        for (int m = team >> 1; m > 0; m >>= 1)
#pragma unroll
            for (int r = 0; r < R; ++r) mean[r] += __shfl_xor_sync(~0u, mean[r], m);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] *= inv;
            m2[r] = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if ((k * team + lane) * V < cg) {
                    vshift<V>(d[r][k], d[r][k], -mean[r]);
                    m2[r] += vdot<V>(d[r][k], d[r][k]);
                }
        }
        for (int m = team >> 1; m > 0; m >>= 1)
#pragma unroll
            for (int r = 0; r < R; ++r) m2[r] += __shfl_xor_sync(~0u, m2[r], m);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!on[r]) continue;
            const long long n = n0 + r * step;
            const float rstd = rsqrtf(fmaf(live[r] ? m2[r] : 0.f, inv, a.eps));
            if (lane == 0) *reinterpret_cast<float2 *>(a.stats + (n * a.G + g) * 2) = make_float2(mean[r], rstd);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * team + lane) * V;
                if (c >= cg) continue;
                float o[V] = {};
                if (live[r]) {
                    float f[V];
                    vscale<V>(f, w[k], rstd);
                    vfma<V>(o, d[r][k], f, b[k]);
                    if (gate != nullptr) {
#pragma unroll
                        for (int u = 0; u < V; ++u) f[u] = q[r][k].at(u);
                        act_of<V>(f, a.act);
                        vmul<V>(o, o, f);
                    } else {
                        act_of<V>(o, a.act);
                    }
                }
                store<V>(y + n * a.C + static_cast<long long>(g) * cg + c, o);
            }
        }
    }
}

// Backward: the sums of dw and db over the rows that a CTA took go to part[blockIdx.x][2][C].
template <typename TX, typename TY, int V, int K, int R>
__global__ void __launch_bounds__(kThr, V * K <= 16 ? 2 : 1) gn_row_backward_kernel(const GnArgs a, int team, float *part) {
    extern __shared__ float red[];  // [rows in flight][dw, db][this CTA's channels]
    const int cg = a.C / a.G;
    const Teams tt = teams_of(a.G, team);
    const int tm = threadIdx.x / team, lane = threadIdx.x & (team - 1);
    const int g = blockIdx.y * tt.gpc + tm % tt.gpc, rr = tm / tt.gpc;
    const bool have = g < a.G && rr < tt.rows;
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
    const long long step = static_cast<long long>(gridDim.x) * tt.rows;
    for (long long n0 = static_cast<long long>(blockIdx.x) * tt.rows + rr; n0 - rr < a.N; n0 += step * R) {
        Raw<TX, V> v[R][K], q[R][K];
        Raw<TY, V> t[R][K];
        bool on[R], live[R];
        float2 st[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const long long n = n0 + r * step;
            on[r] = have && n < a.N;
            live[r] = on[r] && (a.lengths == nullptr || a.lengths[n] > 0);
            st[r] = live[r] ? *reinterpret_cast<const float2 *>(a.stats + (n * a.G + g) * 2) : make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * team + lane) * V;
                v[r][k].zero();
                q[r][k].zero();
                t[r][k].zero();
                if (live[r] && c < cg) {
                    const long long at = n * a.C + static_cast<long long>(g) * cg + c;
                    v[r][k].get(x + at);
                    t[r][k].get(dy + at);
                    if (gate != nullptr) q[r][k].get(gate + at);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const long long base = (n0 + r * step) * a.C + static_cast<long long>(g) * cg;
            const float mean = st[r].x, rstd = st[r].y;
            float xh[K][V], dh[K][V];  // xhat, w dz
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * team + lane) * V;
                float dg[V], z[V], dz[V], slope[V];
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    xh[k][u] = v[r][k].at(u);
                    dz[u] = t[r][k].at(u);  // zero where there is no element
                }
                vshift<V>(xh[k], xh[k], -mean);
                vscale<V>(xh[k], xh[k], rstd);
                vfma<V>(z, xh[k], w[k], b[k]);
                if (gate != nullptr) {
                    float gt[V];
#pragma unroll
                    for (int u = 0; u < V; ++u) gt[u] = q[r][k].at(u);
                    act_and_slope<V>(gt, slope, a.act);
                    vmul<V>(dg, dz, z);
                    vmul<V>(dg, dg, slope);
                    vmul<V>(dz, dz, gt);
                } else {
                    act_and_slope<V>(z, slope, a.act);
                    vmul<V>(dz, dz, slope);
                }
                vadd<V>(db[k], db[k], dz);
                vfma<V>(dw[k], dz, xh[k], dw[k]);
                vmul<V>(dh[k], dz, w[k]);
                s1 += vsum<V>(dh[k]);
                s2 += vdot<V>(dh[k], xh[k]);
                if (gate != nullptr && on[r] && c < cg) store<V>(dgate + base + c, dg);
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
                if (!on[r] || c >= cg) continue;
                float o[V] = {};
                if (live[r]) {
                    // rstd (dh - s1 - xhat s2)
                    vshift<V>(o, dh[k], -s1);
                    float f[V];
                    vscale<V>(f, xh[k], -s2);
                    vadd<V>(o, o, f);
                    vscale<V>(o, o, rstd);
                }
                store<V>(dx + base + c, o);
            }
        }
    }
    // rows in flight summed in order, then this CTA's partial sums out
    const int width = tt.gpc * cg;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * team + lane) * V;
        if (rr < tt.rows && c < cg) {
#pragma unroll
            for (int u = 0; u < V; ++u) {
                red[(rr * 2 + 0) * width + (tm % tt.gpc) * cg + c + u] = dw[k][u];
                red[(rr * 2 + 1) * width + (tm % tt.gpc) * cg + c + u] = db[k][u];
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * width; i += kThr) {
        const int which = i / width, c = i % width, ch = blockIdx.y * width + c;
        if (ch >= a.C) continue;
        float s = 0.f;
        for (int q = 0; q < tt.rows; ++q) s += red[(q * 2 + which) * width + c];
        part[(static_cast<long long>(blockIdx.x) * 2 + which) * a.C + ch] = s;
    }
}

// dw, db [C] = sums of part [rows][2][C], a block for 32 channels of one of them: a slice of the rows per warp, each
// in row order, then the slices in order
__device__ __forceinline__ void param_sum(int block, const float *__restrict__ part, int rows, int C, float *dw, float *db) {
    __shared__ float red[32][33];
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int c = (block >> 1) * 32 + lane, which = block & 1;
    float s = 0.f;
    if (c < C) {
#pragma unroll 8
        for (int r = sl; r < rows; r += warps) s += part[(static_cast<long long>(r) * 2 + which) * C + c];
    }
    red[sl][lane] = s;
    __syncthreads();
    if (sl == 0 && c < C) {
        for (int q = 1; q < warps; ++q) s += red[q][lane];
        float *out = which == 0 ? dw : db;
        if (out != nullptr) out[c] = s;
    }
}
int param_blocks(int C) { return (C + 31) / 32 * 2; }
__global__ void __launch_bounds__(1024) gn_param_sum_kernel(const float *part, int rows, int C, float *dw, float *db) {
    param_sum(blockIdx.x, part, rows, C, dw, db);
}

// ---- statistics over a sequence ------------------------------------------------------------------------------

// A CTA takes `rows` rows of one n.  Its threads span the channels (vectors of V within one group) and, where
// there are fewer vectors than threads, several rows at once.
struct Span {
    int cols, par;  // vectors per row; rows in flight
};
template <int V>
__host__ __device__ __forceinline__ Span span_of(const GnArgs &a) {
    const int cols = a.C / V;
    return {cols, cols >= kThr ? 1 : kThr / cols};
}
// threads of such a CTA
template <int V>
int threads_of(const GnArgs &a) {
    const Span sp = span_of<V>(a);
    return sp.par == 1 && sp.cols >= kThr ? kThr : (sp.cols * sp.par + 31) / 32 * 32;
}

// part[n][chunk][g] = moments of group g in this CTA's rows
template <typename TX, int V>
__global__ void __launch_bounds__(kThr) gn_stats_kernel(const GnArgs a, int rows, int chunks, Moments *part) {
    constexpr int RB = 32 / V < 8 ? 32 / V : 8;  // rows a thread holds at a time
    __shared__ Moments red[kThr];
    extern __shared__ Moments acc[];  // [G]
    const int n = static_cast<int>(blockIdx.x / chunks), ch = static_cast<int>(blockIdx.x % chunks), L = row_count(a, n);
    // rows are counted from the block's first one: counters step past the last row, and S may be 2^31 - 1
    const long long lo = static_cast<long long>(ch) * rows;
    const int count = lo < L ? static_cast<int>(min(static_cast<long long>(rows), L - lo)) : 0;
    const TX *x = static_cast<const TX *>(a.x) + (static_cast<long long>(n) * a.S + lo) * a.C;
    const Span sp = span_of<V>(a);
    const int cg = a.C / a.G, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int g = threadIdx.x; g < a.G; g += blockDim.x) acc[g] = {0.f, 0.f, 0.f};
    for (int cb = 0; cb < sp.cols; cb += kThr) {
        const int width = min(kThr, sp.cols - cb);
        const int r0 = sp.par == 1 ? 0 : threadIdx.x / sp.cols;
        const int col = sp.par == 1 ? threadIdx.x : threadIdx.x % sp.cols;
        Moments m = {0.f, 0.f, 0.f};
        if (col < width && r0 < sp.par) {
            const TX *p = x + static_cast<long long>(cb + col) * V;
            for (int s = r0; s < count; s += RB * sp.par) {
                float v[RB][V];
                int cnt = 0;
                float sum = 0.f;
#pragma unroll
                for (int u = 0; u < RB; ++u)
                    if (s + u * sp.par < count) {
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
        for (int g = g_lo + warp; g <= g_hi; g += blockDim.x / 32) {
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
    for (int g = threadIdx.x; g < a.G; g += blockDim.x) out[g] = acc[g];
}

// A warp joins the moments of one (n, group) over the chunks, `step` apart: mean and 1 / sqrt(var + eps)
__device__ __forceinline__ float2 join_chunks(const Moments *p, int chunks, int step, float eps, int lane) {
    Moments t = {0.f, 0.f, 0.f};
    for (int q = lane; q < chunks; q += 32) t = join(t, p[static_cast<long long>(q) * step]);
#pragma unroll
    for (int q = 16; q > 0; q >>= 1) t = join(t, shuffle_xor(t, q));
    return make_float2(t.mean, rsqrtf((t.n > 0.f ? t.m2 / t.n : 0.f) + eps));
}

__global__ void __launch_bounds__(kThr) gn_stats_join_kernel(const GnArgs a, int chunks, const Moments *part) {
    const long long i = (static_cast<long long>(blockIdx.x) * kThr + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (i >= static_cast<long long>(a.N) * a.G) return;
    const float2 st = join_chunks(part + i / a.G * chunks * a.G + i % a.G, chunks, a.G, a.eps, lane);
    if (lane == 0) *reinterpret_cast<float2 *>(a.stats + i * 2) = st;
}

// The second pass over x.  JOIN: every CTA joins its n's partial statistics by itself, a warp per group, where they are
// few enough that this costs less than a launch of its own (gn_stats_join_kernel).  Blocks in reversed order, from what
// the first pass read last, are no gain here (129.1 us both on [16, 65536, 64] fp32 to bf16, 73.8 on half of it).
template <typename TX, typename TY, int V, bool JOIN>
__global__ void __launch_bounds__(kThr) gn_apply_kernel(const GnArgs a, int rows, int chunks, const Moments *part) {
    extern __shared__ float2 joined[];  // [G]
    const int n = static_cast<int>(blockIdx.x / chunks), ch = static_cast<int>(blockIdx.x % chunks), L = row_count(a, n);
    const long long lo = static_cast<long long>(ch) * rows;
    // rows counted from the block's first one, as in gn_stats_kernel: `count` of them, the first `live` within the length
    const int count = static_cast<int>(min(static_cast<long long>(rows), a.S - lo));
    const int live = static_cast<int>(L - lo);
    const long long nb = (static_cast<long long>(n) * a.S + lo) * a.C;
    const TX *x = static_cast<const TX *>(a.x) + nb;
    const TX *gate = a.gate == nullptr ? nullptr : static_cast<const TX *>(a.gate) + nb;
    TY *y = static_cast<TY *>(a.y) + nb;
    const Span sp = span_of<V>(a);
    if (JOIN) {
        const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
        for (int g = threadIdx.x >> 5; g < a.G; g += warps) {
            const float2 st = join_chunks(part + static_cast<long long>(n) * chunks * a.G + g, chunks, a.G, a.eps, lane);
            if (lane == 0) {
                joined[g] = st;
                if (ch == 0) *reinterpret_cast<float2 *>(a.stats + (static_cast<long long>(n) * a.G + g) * 2) = st;
            }
        }
        __syncthreads();
    }
    const float2 *stats = JOIN ? joined : reinterpret_cast<const float2 *>(a.stats) + static_cast<long long>(n) * a.G;
    const int r0 = sp.par == 1 ? 0 : threadIdx.x / sp.cols;
    if (r0 >= sp.par) return;
    for (int col = sp.par == 1 ? threadIdx.x : threadIdx.x % sp.cols; col < sp.cols; col += sp.par == 1 ? kThr : sp.cols) {
        const int c = col * V, g = c / (a.C / a.G);
        const float2 st = stats[g];
        float w[V], b[V];
        load_wb<V>(a, c, w, b);
#pragma unroll
        for (int i = 0; i < V; ++i) {  // z = x * w' + b'' after the mean is taken off
            w[i] *= st.y;
        }
#pragma unroll 4
        for (int s = r0; s < count; s += sp.par) {
            const long long at = static_cast<long long>(s) * a.C + c;
            float o[V] = {};
            if (s < live) {
                float v[V], q[V];
                load<V>(x + at, v);
                if (gate != nullptr) load<V>(gate + at, q);
                vshift<V>(v, v, -st.x);
                vfma<V>(o, v, w, b);
                if (gate != nullptr) {
                    act_of<V>(q, a.act);
                    vmul<V>(o, o, q);
                } else {
                    act_of<V>(o, a.act);
                }
            }
            store<V>(y + at, o);
        }
    }
}

// From x, dy and the gate's values q to xhat (in v), dz (in t) and, with a gate, dgate (in q)
template <int V, bool GATE>
__device__ __forceinline__ void dz_of(const GnArgs &a, float2 st, const float (&w)[V], const float (&b)[V], float (&v)[V],
                                      float (&t)[V], float (&q)[V]) {
    float z[V], slope[V];
    vshift<V>(v, v, -st.x);
    vscale<V>(v, v, st.y);
    vfma<V>(z, v, w, b);
    if constexpr (GATE) {
        act_and_slope<V>(q, slope, a.act);
        vmul<V>(z, z, t);
        vmul<V>(t, t, q);
        vmul<V>(q, z, slope);
    } else {
        act_and_slope<V>(z, slope, a.act);
        vmul<V>(t, t, slope);
    }
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
                dz_of<V, GATE>(a, st, w, b, v, t, q);
                vadd<V>(db, db, t);
                vfma<V>(dw, t, v, dw);
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
            for (int i = threadIdx.x; i < 2 * a.C; i += blockDim.x) {
                const int which = i / a.C, c = i % a.C;
                float s = 0.f;
                for (int q = 0; q < sp.par; ++q) s += red[which][q * a.C + c];
                out[i] = s;
            }
        }
    }
}

// A CTA takes one (n, group) after another, as N G may pass what a grid holds: channel sums over the chunks ->
// chan[n][2][C], group sums of w dz and w dz xhat -> gsum[n][g][2].  Threads span the group's channels and, where those
// are few, slices of the chunks.
__global__ void __launch_bounds__(kThr) gn_channel_join_kernel(const GnArgs a, int chunks, const float *__restrict__ part,
                                                               float *chan, float *gsum) {
    __shared__ float red[2][kThr];
    const int cg = a.C / a.G, cols = min(cg, kThr), slices = kThr / cols;
    const int col = threadIdx.x % cols, sl = threadIdx.x / cols;
    for (long long i = blockIdx.x; i < static_cast<long long>(a.N) * a.G; i += gridDim.x) {
        const int n = static_cast<int>(i / a.G), g = static_cast<int>(i % a.G);
        const float *p = part + static_cast<long long>(n) * chunks * 2 * a.C + g * cg;
        float *ch = chan + static_cast<long long>(n) * 2 * a.C + g * cg;
        float s1 = 0.f, s2 = 0.f;  // w dz, w dz xhat of this thread's channels
        for (int c0 = 0; c0 < cg; c0 += cols) {
            const int c = c0 + col;
            float dw = 0.f, db = 0.f;
            if (c < cg && sl < slices) {
#pragma unroll 4
                for (int q = sl; q < chunks; q += slices) {
                    dw += p[static_cast<long long>(q) * 2 * a.C + c];
                    db += p[static_cast<long long>(q) * 2 * a.C + a.C + c];
                }
            }
            __syncthreads();
            red[0][threadIdx.x] = dw, red[1][threadIdx.x] = db;
            __syncthreads();
            if (c < cg && sl == 0) {
                for (int q = 1; q < slices; ++q) dw += red[0][q * cols + col], db += red[1][q * cols + col];
                ch[c] = dw, ch[a.C + c] = db;
                const float w = a.weight != nullptr ? a.weight[g * cg + c] : 1.f;
                s1 = fmaf(w, db, s1), s2 = fmaf(w, dw, s2);
            }
        }
        __syncthreads();
        red[0][threadIdx.x] = s1, red[1][threadIdx.x] = s2;
        __syncthreads();
        for (int m = kThr / 2; m > 0; m >>= 1) {
            if (threadIdx.x < m)
                red[0][threadIdx.x] += red[0][threadIdx.x + m], red[1][threadIdx.x] += red[1][threadIdx.x + m];
            __syncthreads();
        }
        if (threadIdx.x == 0) *reinterpret_cast<float2 *>(gsum + i * 2) = make_float2(red[0][0], red[1][0]);
    }
}

template <typename TX, typename TY, int V, bool GATE>
__global__ void __launch_bounds__(kThr) gn_backward_apply_kernel(const GnArgs a, int rows, int chunks, const float *gsum,
                                                                 const float *chan) {
    const unsigned blocks = static_cast<unsigned>(chunks) * a.N;
    if (blockIdx.x >= blocks) {  // the parameters' gradients
        param_sum(blockIdx.x - blocks, chan, a.N, a.C, a.dweight, a.dbias);
        return;
    }
    // in reversed order: some of what the first pass read last is still in L2 ([16, 32768, 64] fp32 to bf16: 133 against
    // 135 us, [8, 16384, 128] fp32 86 against 88; no difference on inputs of twice that size)
    const unsigned bid = blocks - 1 - blockIdx.x;
    const int n = static_cast<int>(bid / chunks), ch = static_cast<int>(bid % chunks), L = row_count(a, n);
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
            float o[V] = {}, q[V] = {};
            if (s < L) {
                float v[V], t[V];
                load<V>(x + at, v);
                load<V>(dy + at, t);
                if (GATE) load<V>(gate + at, q);
                dz_of<V, GATE>(a, st, w, b, v, t, q);
                // r (w dz - gs.x - xhat gs.y)
                vmul<V>(o, w, t);
                vshift<V>(o, o, -gs.x);
                vscale<V>(v, v, -gs.y);
                vadd<V>(o, o, v);
                vscale<V>(o, o, st.y);
            }
            store<V>(dx + at, o);
            if (GATE) store<V>(dgate + at, q);
        }
    }
}

// ---- plans and dispatch --------------------------------------------------------------------------------------

constexpr int kJoinMost = 1024;  // partial moments of one n that every CTA of the second pass joins by itself
constexpr long long kJoinGrid = 1 << 20;  // CTAs of gn_channel_join_kernel, at most
// channels of a group that a warp holds, 32 per lane: in registers forward; the backward kernels of 16 and 32 per lane
// also use local memory (up to 268 bytes a thread)
constexpr int kRowMost = 1024;

bool row_regime(const GnArgs &a) { return a.S == 1 && a.C / a.G <= kRowMost; }
int vec_of(const GnArgs &a) {
    const int cg = a.C / a.G;
    return cg % 8 == 0 ? 8 : cg % 4 == 0 ? 4 : 1;
}
// vectors that a lane holds of a group: more than one where 32 lanes would not hold it, and in the forward pass two
// where a group has them, which halves the shuffles per element ([32768, 16 x 128] bf16 gated: 108 -> 96 us; the
// backward pass has no registers for it: 61 -> 66 us on 8192 rows)
int vectors_of(const GnArgs &a, bool backward) {
    const int cg = a.C / a.G, V = vec_of(a);
    if (V == 8) return cg <= 8 || (backward && cg <= 256) ? 1 : cg <= 512 ? 2 : 4;
    if (V == 4) return cg <= 128 ? 1 : 8;
    return cg <= 128 ? 4 : 32;
}
int team_of(const GnArgs &a, bool backward) {
    const int per = vec_of(a) * vectors_of(a, backward), need = (a.C / a.G + per - 1) / per;
    int t = 1;
    while (t < need && t < 32) t *= 2;
    return t;
}
// rows per CTA: forward 4 CTAs of 256 threads per SM, as many as run at once (8: [16, 65536, 64] 139 against 129 us),
// backward 8 (ragged [8, 1000, 640] 41 against 49 us with 4); at least about 4K elements each.  N S is below 2^31, so that a
// block has at most 3.7e6 rows and its kernel counts them in 32 bits
int chunk_rows(const GnArgs &a, bool backward) {
    const long long all = static_cast<long long>(a.N) * a.S, ctas = 148 * (backward ? 8 : 4);
    long long rows = (all + ctas - 1) / ctas;
    const long long least = (4096 + a.C - 1) / a.C;
    if (rows < least) rows = least;
    if (rows > a.S) rows = a.S;
    return static_cast<int>(rows);
}
// blocks of `rows` rows in one n; S + rows may pass 32 bits
int chunks_of(const GnArgs &a, int rows) { return static_cast<int>((static_cast<long long>(a.S) + rows - 1) / rows); }
// CTAs along the rows: `per_sm` of them per SM, if there are that many rows
int row_ctas(const GnArgs &a, int per_sm, bool backward) {
    const int per = kThr / team_of(a, backward), gpc = per < a.G ? per : a.G, rows = per / gpc;
    const int by = (a.G + gpc - 1) / gpc;
    long long bx = (148 * per_sm + by - 1) / by;
    const long long most = (static_cast<long long>(a.N) + rows - 1) / rows;
    if (bx > most) bx = most;
    return static_cast<int>(bx < 1 ? 1 : bx);
}
size_t al(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// rows in flight per team
template <int V, int K>
constexpr int rows_held(bool backward) {
    return V * K <= (backward ? 8 : 16) ? 2 : 1;
}

template <typename TX, typename TY, int V, int K>
cudaError_t row_forward(const GnArgs &a, cudaStream_t s) {
    const int team = team_of(a, false), per = kThr / team, gpc = per < a.G ? per : a.G;
    const dim3 grid(row_ctas(a, 8, false), (a.G + gpc - 1) / gpc);
    gn_row_forward_kernel<TX, TY, V, K, rows_held<V, K>(false)><<<grid, kThr, 0, s>>>(a, team);
    return cudaGetLastError();
}

template <typename TX, typename TY, int V, int K>
cudaError_t row_backward(const GnArgs &a, cudaStream_t s) {
    const int team = team_of(a, true), per = kThr / team, gpc = per < a.G ? per : a.G, rows = per / gpc;
    const int bx = row_ctas(a, 4, true);
    const dim3 grid(bx, (a.G + gpc - 1) / gpc);
    const int smem = rows * 2 * gpc * (a.C / a.G) * 4;
    auto k = gn_row_backward_kernel<TX, TY, V, K, rows_held<V, K>(true)>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    k<<<grid, kThr, smem, s>>>(a, team, reinterpret_cast<float *>(a.ws));
    gn_param_sum_kernel<<<param_blocks(a.C), 1024, 0, s>>>(reinterpret_cast<float *>(a.ws), bx, a.C, a.dweight, a.dbias);
    return cudaGetLastError();
}

template <typename TX, typename TY, int V>
cudaError_t seq_forward(const GnArgs &a, cudaStream_t s) {
    const int rows = chunk_rows(a, false), chunks = chunks_of(a, rows);
    Moments *part = reinterpret_cast<Moments *>(a.ws);
    const unsigned grid = static_cast<unsigned>(chunks) * a.N;
    gn_stats_kernel<TX, V><<<grid, threads_of<V>(a), a.G * sizeof(Moments), s>>>(a, rows, chunks, part);
    if (static_cast<long long>(chunks) * a.G <= kJoinMost) {
        gn_apply_kernel<TX, TY, V, true><<<grid, threads_of<V>(a), a.G * sizeof(float2), s>>>(a, rows, chunks, part);
    } else {
        const long long warps = static_cast<long long>(a.N) * a.G;
        gn_stats_join_kernel<<<static_cast<unsigned>((warps * 32 + kThr - 1) / kThr), kThr, 0, s>>>(a, chunks, part);
        gn_apply_kernel<TX, TY, V, false><<<grid, threads_of<V>(a), 0, s>>>(a, rows, chunks, part);
    }
    return cudaGetLastError();
}

template <typename TX, typename TY, int V, bool GATE>
cudaError_t seq_backward_g(const GnArgs &a, cudaStream_t s) {
    const int rows = chunk_rows(a, true), chunks = chunks_of(a, rows);
    const unsigned grid = static_cast<unsigned>(chunks) * a.N;
    float *part = reinterpret_cast<float *>(a.ws);
    float *chan = reinterpret_cast<float *>(a.ws + al(static_cast<size_t>(a.N) * chunks * 2 * a.C * 4));
    float *gsum = reinterpret_cast<float *>(reinterpret_cast<char *>(chan) + al(static_cast<size_t>(a.N) * 2 * a.C * 4));
    gn_channel_sum_kernel<TX, TY, V, GATE><<<grid, threads_of<V>(a), 0, s>>>(a, rows, chunks, part);
    const long long joins = static_cast<long long>(a.N) * a.G;
    gn_channel_join_kernel<<<static_cast<unsigned>(joins < kJoinGrid ? joins : kJoinGrid), kThr, 0, s>>>(a, chunks, part, chan,
                                                                                                        gsum);
    // few rows to sum: blocks of the same launch do it
    const bool with = a.N <= 256;
    gn_backward_apply_kernel<TX, TY, V, GATE>
        <<<grid + (with ? param_blocks(a.C) : 0), threads_of<V>(a), 0, s>>>(a, rows, chunks, gsum, chan);
    if (!with) gn_param_sum_kernel<<<param_blocks(a.C), 1024, 0, s>>>(chan, a.N, a.C, a.dweight, a.dbias);
    return cudaGetLastError();
}

template <typename TX, typename TY, bool BACK>
cudaError_t dispatch(const GnArgs &a, cudaStream_t s) {
    const int V = vec_of(a);
    if (row_regime(a)) {
        const int K = vectors_of(a, BACK);
        if (BACK) {
            if (V == 8)
                return K == 1   ? row_backward<TX, TY, 8, 1>(a, s)
                       : K == 2 ? row_backward<TX, TY, 8, 2>(a, s)
                                : row_backward<TX, TY, 8, 4>(a, s);
            if (V == 4) return K == 1 ? row_backward<TX, TY, 4, 1>(a, s) : row_backward<TX, TY, 4, 8>(a, s);
            return K == 4 ? row_backward<TX, TY, 1, 4>(a, s) : row_backward<TX, TY, 1, 32>(a, s);
        }
        if (V == 8)
            return K == 1   ? row_forward<TX, TY, 8, 1>(a, s)
                   : K == 2 ? row_forward<TX, TY, 8, 2>(a, s)
                            : row_forward<TX, TY, 8, 4>(a, s);
        if (V == 4) return K == 1 ? row_forward<TX, TY, 4, 1>(a, s) : row_forward<TX, TY, 4, 8>(a, s);
        return K == 4 ? row_forward<TX, TY, 1, 4>(a, s) : row_forward<TX, TY, 1, 32>(a, s);
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
        return backward ? al(static_cast<size_t>(row_ctas(a, 4, true)) * 2 * a.C * 4) : 0;
    const int rows = chunk_rows(a, backward), chunks = chunks_of(a, rows);
    if (!backward) return al(static_cast<size_t>(a.N) * chunks * a.G * sizeof(Moments));
    return al(static_cast<size_t>(a.N) * chunks * 2 * a.C * 4) + al(static_cast<size_t>(a.N) * 2 * a.C * 4) +
           al(static_cast<size_t>(a.N) * a.G * 8);
}

cudaError_t launch_gn_forward(const GnArgs &a, cudaStream_t s) { return by_type<false>(a, s); }
cudaError_t launch_gn_backward(const GnArgs &a, cudaStream_t s) { return by_type<true>(a, s); }

}  // namespace pararnn
