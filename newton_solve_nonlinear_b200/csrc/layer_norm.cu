// layer_norm.cu -- the norm of a residual stream, forward and backward (sm_100a).
//
//   r = residual + x,   m = mean of r's row (0 for the rms form),   k = 1 / sqrt(mean (r - m)^2 + eps),
//   y = (r - m) k weight + bias
//   dr = k (u - mean(u) - h mean(u h)) + dr_in with u = dy weight, h = (r - m) k (without mean(u) in the rms form),
//   dweight = sum over the rows of dy h,  dbias = sum of dy
//
// A row lives in the registers of a team of 32, 256 or 1024 threads, so that it is read once and its variance is formed
// about its mean; longer rows (more than 32768 channels, 8192 off alignment) are read again.
// Bound by HBM: 32768 rows of 2048, bf16 onto an fp32 stream, 129 us, 0.95 of its rate; backward 16384 rows 108 us, 0.75.
// With more than four vectors to a thread registers run short: backward rows of 4096 and 8192 channels, one or two CTAs to an
// SM, move at 0.50 and 0.54 of HBM's rate, and rows of 8193 to 32768 aligned channels go through local memory in part (16384:
// forward 0.65, backward 0.08).
#include <algorithm>

#include "layer_norm.cuh"
#include "rows.cuh"

namespace pararnn {
using namespace rows;
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// The sums of a and b over a team's threads, to all of them.  s: a pair per warp of the CTA, twice, used in turn (`turn`
// counts the calls): one barrier is enough, as the next call writes elsewhere.
template <int TEAM>
__device__ __forceinline__ float2 team_sum(float a, float b, float2 (*s)[32], int &turn) {
    a = warp_sum(a), b = warp_sum(b);
    if constexpr (TEAM > 32) {
        float2 *at = s[turn++ & 1];
        if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const float2 v = (threadIdx.x & 31) < TEAM / 32 ? at[threadIdx.x & 31] : make_float2(0.f, 0.f);
        a = warp_sum(v.x), b = warp_sum(v.y);
    }
    return make_float2(a, b);
}
template <int TEAM>
__device__ __forceinline__ float team_sum(float a, float2 (*s)[32], int &turn) {
    return team_sum<TEAM>(a, 0.f, s, turn).x;
}

// K vectors of a row, `step` vectors apart, n of them in all: first as they lie in memory, so that nothing waits for a load
// before all are under way; the branch on the type stands outside the loop for the same reason.
template <int V>
struct Bits {
    unsigned w[V];
};
template <int V, int K>
__device__ __forceinline__ void fetch(const void *p, long long base, bool f32, int at, int step, int n, Bits<V> (&r)[K]) {
    if (f32) {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const float *q = static_cast<const float *>(p) + base + (at + i * step) * V;
            if (at + i * step >= n) continue;
            if constexpr (V == 4) {
                const uint4 x = *reinterpret_cast<const uint4 *>(q);
                r[i].w[0] = x.x, r[i].w[1] = x.y, r[i].w[2] = x.z, r[i].w[3] = x.w;
            } else {
                r[i].w[0] = *reinterpret_cast<const unsigned *>(q);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p) + base + (at + i * step) * V;
            if (at + i * step >= n) continue;
            if constexpr (V == 4) {
                const uint2 x = *reinterpret_cast<const uint2 *>(q);
                r[i].w[0] = x.x, r[i].w[1] = x.y;
            } else {
                r[i].w[0] = *reinterpret_cast<const unsigned short *>(q);
            }
        }
    }
}
template <int V, int K>
__device__ __forceinline__ void values(const Bits<V> (&r)[K], bool f32, float (&v)[K][V]) {
    if (f32) {
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int u = 0; u < V; ++u) v[i][u] = __uint_as_float(r[i].w[u]);
    } else {
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int u = 0; u < V; ++u) v[i][u] = __uint_as_float(u % 2 == 0 ? r[i].w[u / 2] << 16 : r[i].w[u / 2] & 0xffff0000u);
    }
}
template <int V, int K>
__device__ __forceinline__ void store_all(void *p, long long base, bool f32, int at, int step, int n, const float (&v)[K][V]) {
    if (f32) {
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (at + i * step < n) store<V>(static_cast<float *>(p) + base + (at + i * step) * V, v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (at + i * step < n) store<V>(static_cast<__nv_bfloat16 *>(p) + base + (at + i * step) * V, v[i]);
    }
}

template <int TEAM>
constexpr int cta_of() { return TEAM > 256 ? TEAM : 256; }

// K vectors of V channels per thread; K = 0: rows of any length, read again for each pass
template <int V, int TEAM, int K>
__global__ void __launch_bounds__(cta_of<TEAM>()) ln_forward_kernel(const LnArgs w) {
    constexpr int TEAMS = cta_of<TEAM>() / TEAM;
    __shared__ float2 s_sum[2][32];
    int turn = 0;
    const int lane = threadIdx.x % TEAM, nv = w.C / V;
    const long long rows = static_cast<long long>(w.N) * w.S;
    const long long row = static_cast<long long>(blockIdx.x) * TEAMS + threadIdx.x / TEAM;
    if (row >= rows) return;  // whole warps where TEAM is 32, whole CTAs otherwise
    const bool xf = w.x_dtype == PARARNN_F32, rf = w.r_dtype == PARARNN_F32, yf = w.y_dtype == PARARNN_F32;
    const bool on = row % w.S < count(w.lengths, static_cast<int>(row / w.S), w.S);
    const long long base = row * w.C;
    const float per = 1.f / w.C;
    auto read = [&](int c, float (&v)[V]) {
#pragma unroll
        for (int u = 0; u < V; ++u) v[u] = 0.f;
        if (!on) return;
        load<V>(w.x, base + c, xf, v);
        if (w.residual != nullptr) {
            float q[V];
            load<V>(w.residual, base + c, rf, q);
#pragma unroll
            for (int u = 0; u < V; ++u) v[u] += q[u];
        }
    };
    auto write = [&](int c, const float (&v)[V], float m, float k) {
        if (w.r != nullptr) store<V>(w.r, base + c, rf, v);
        float g[V], o[V];
#pragma unroll
        for (int u = 0; u < V; ++u) o[u] = (v[u] - m) * k;
        if (w.weight != nullptr) {
            load<V>(w.weight + c, g);
#pragma unroll
            for (int u = 0; u < V; ++u) o[u] *= g[u];
        }
        if (w.bias != nullptr) {
            load<V>(w.bias + c, g);
#pragma unroll
            for (int u = 0; u < V; ++u) o[u] += g[u];
        }
        if (!on) {
#pragma unroll
            for (int u = 0; u < V; ++u) o[u] = 0.f;
        }
        store<V>(w.y, base + c, yf, o);
    };
    float m = 0.f, k;
    if constexpr (K > 0) {
        float v[K][V], sum = 0.f;
        {
            Bits<V> rx[K] = {}, rr[K] = {};
            const int n = on ? nv : 0;
            fetch(w.x, base, xf, lane, TEAM, n, rx);
            if (w.residual != nullptr) fetch(w.residual, base, rf, lane, TEAM, n, rr);
            values(rx, xf, v);
            if (w.residual != nullptr) {
                float q[K][V];
                values(rr, rf, q);
#pragma unroll
                for (int i = 0; i < K; ++i)
#pragma unroll
                    for (int u = 0; u < V; ++u) v[i][u] += q[i][u];
            }
        }
        if (w.r != nullptr) store_all(w.r, base, rf, lane, TEAM, nv, v);
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int u = 0; u < V; ++u) sum += v[i][u];
        if (!w.rms) m = team_sum<TEAM>(sum, s_sum, turn) * per;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (lane + i * TEAM < nv) {
#pragma unroll
                for (int u = 0; u < V; ++u) v[i][u] -= m, sum = fmaf(v[i][u], v[i][u], sum);
            }
        k = rsqrtf(team_sum<TEAM>(sum, s_sum, turn) * per + w.eps);
        const float scale = on ? k : 0.f;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            if (lane + i * TEAM >= nv) continue;
            const int c = (lane + i * TEAM) * V;
            float g[V], o[V];
#pragma unroll
            for (int u = 0; u < V; ++u) g[u] = 1.f, o[u] = 0.f;
            // neither where the row does not count: it is zero whatever they hold
            if (w.weight != nullptr && on) load<V>(w.weight + c, g);
            if (w.bias != nullptr && on) load<V>(w.bias + c, o);
#pragma unroll
            for (int u = 0; u < V; ++u) v[i][u] = fmaf(v[i][u] * scale, g[u], o[u]);
        }
        store_all(w.y, base, yf, lane, TEAM, nv, v);
    } else {
        float v[V], sum = 0.f;
        if (!w.rms) {
            for (int at = lane; at < nv; at += TEAM) {
                read(at * V, v);
#pragma unroll
                for (int u = 0; u < V; ++u) sum += v[u];
            }
            m = team_sum<TEAM>(sum, s_sum, turn) * per;
        }
        sum = 0.f;
        for (int at = lane; at < nv; at += TEAM) {
            read(at * V, v);
#pragma unroll
            for (int u = 0; u < V; ++u) sum = fmaf(v[u] - m, v[u] - m, sum);
        }
        k = rsqrtf(team_sum<TEAM>(sum, s_sum, turn) * per + w.eps);
        for (int at = lane; at < nv; at += TEAM) {
            read(at * V, v);
            write(at * V, v, m, k);
        }
    }
    if (lane == 0) *reinterpret_cast<float2 *>(w.stats + 2 * row) = make_float2(m, k);
}

// A CTA takes every gridDim.x-th group of rows and keeps its sums for the weight and the bias in registers; K = 0 leaves
// these to ln_columns_kernel.
template <int V, int TEAM, int K>
__global__ void __launch_bounds__(cta_of<TEAM>()) ln_backward_kernel(const LnArgs w) {
    constexpr int TEAMS = cta_of<TEAM>() / TEAM, KK = K > 0 ? K : 1;
    __shared__ float2 s_sum[2][32];
    int turn = 0;
    extern __shared__ float s_part[];  // TEAM = 32: [8][2 C]
    const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM, nv = w.C / V;
    const long long rows = static_cast<long long>(w.N) * w.S;
    const bool xf = w.x_dtype == PARARNN_F32, rf = w.r_dtype == PARARNN_F32, yf = w.y_dtype == PARARNN_F32;
    const float per = 1.f / w.C;
    float dw[KK][V] = {}, db[KK][V] = {};
    // u = dy weight and h of V channels; zero where the row does not count
    auto read = [&](long long base, int c, float m, float k, float (&u)[V], float (&h)[V], float (&dy)[V]) {
        load<V>(w.r, base + c, rf, h);
        load<V>(w.y, base + c, yf, dy);
        float g[V];
        if (w.weight != nullptr) {
            load<V>(w.weight + c, g);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) g[j] = 1.f;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = (h[j] - m) * k, u[j] = dy[j] * g[j];
    };
    auto write = [&](long long base, int c, float k, float mu, float muh, const float (&u)[V], const float (&h)[V]) {
        float o[V];
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = k * (u[j] - mu - h[j] * muh);
        if (w.dr_in != nullptr) {
            float q[V];
            load<V>(w.dr_in, base + c, rf, q);
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] += q[j];
        }
        store<V>(w.dr, base + c, rf, o);
        if (w.dx != nullptr) store<V>(w.dx, base + c, xf, o);
    };
    for (long long row = static_cast<long long>(blockIdx.x) * TEAMS + team; row < rows;
         row += static_cast<long long>(gridDim.x) * TEAMS) {
        const long long base = row * w.C;
        if (row % w.S >= count(w.lengths, static_cast<int>(row / w.S), w.S)) {
            const float zero[V] = {};
            for (int at = lane; at < nv; at += TEAM) {
                store<V>(w.dr, base + at * V, rf, zero);
                if (w.dx != nullptr) store<V>(w.dx, base + at * V, xf, zero);
            }
            continue;
        }
        const float m = w.stats[2 * row], k = w.stats[2 * row + 1];
        float su = 0.f, suh = 0.f;
        if constexpr (K > 0) {
            float u[K][V], h[K][V], dys[K][V];
            Bits<V> ri[K];
            {
                Bits<V> rr[K], ry[K];
                fetch(w.r, base, rf, lane, TEAM, nv, rr);
                fetch(w.y, base, yf, lane, TEAM, nv, ry);
                if (w.dr_in != nullptr) fetch(w.dr_in, base, rf, lane, TEAM, nv, ri);
                values(rr, rf, h), values(ry, yf, dys);
            }
#pragma unroll
            for (int i = 0; i < K; ++i) {
                const int at = lane + i * TEAM;
                if (at >= nv) continue;
                const float(&dy)[V] = dys[i];
                float g[V];
#pragma unroll
                for (int j = 0; j < V; ++j) g[j] = 1.f;
                if (w.weight != nullptr) load<V>(w.weight + at * V, g);
#pragma unroll
                for (int j = 0; j < V; ++j) h[i][j] = (h[i][j] - m) * k, u[i][j] = dy[j] * g[j];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    su += u[i][j], suh = fmaf(u[i][j], h[i][j], suh);
                    dw[i][j] = fmaf(dy[j], h[i][j], dw[i][j]), db[i][j] += dy[j];
                }
            }
            const float2 sums = team_sum<TEAM>(su, suh, s_sum, turn);
            su = w.rms ? 0.f : sums.x * per, suh = sums.y * per;
#pragma unroll
            for (int i = 0; i < K; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) u[i][j] = k * (u[i][j] - su - h[i][j] * suh);
            if (w.dr_in != nullptr) {
                values(ri, rf, h);
#pragma unroll
                for (int i = 0; i < K; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) u[i][j] += h[i][j];
            }
            store_all(w.dr, base, rf, lane, TEAM, nv, u);
            if (w.dx != nullptr) store_all(w.dx, base, xf, lane, TEAM, nv, u);
        } else {
            float u[V], h[V], dy[V];
            for (int at = lane; at < nv; at += TEAM) {
                read(base, at * V, m, k, u, h, dy);
#pragma unroll
                for (int j = 0; j < V; ++j) su += u[j], suh = fmaf(u[j], h[j], suh);
            }
            const float2 sums = team_sum<TEAM>(su, suh, s_sum, turn);
            su = w.rms ? 0.f : sums.x * per, suh = sums.y * per;
            for (int at = lane; at < nv; at += TEAM) {
                read(base, at * V, m, k, u, h, dy);
                write(base, at * V, k, su, suh, u, h);
            }
        }
    }
    if constexpr (K > 0) {
        float *part = w.part + static_cast<long long>(blockIdx.x) * 2 * w.C;
        float *to = TEAMS > 1 ? s_part + team * 2 * w.C : part;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int at = lane + i * TEAM;
            if (at >= nv) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) to[at * V + j] = dw[i][j], to[w.C + at * V + j] = db[i][j];
        }
        if constexpr (TEAMS > 1) {
            __syncthreads();
            for (int c = threadIdx.x; c < 2 * w.C; c += cta_of<TEAM>()) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < TEAMS; ++i) sum += s_part[i * 2 * w.C + c];
                part[c] = sum;
            }
        }
    }
}

// dweight and dbias of rows too long for registers: a CTA takes 32 columns of every gridDim.y-th row
__global__ void __launch_bounds__(256) ln_columns_kernel(const LnArgs w) {
    __shared__ float s[2][8][32];
    const int lane = threadIdx.x % 32, y = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    const long long rows = static_cast<long long>(w.N) * w.S;
    const bool rf = w.r_dtype == PARARNN_F32, yf = w.y_dtype == PARARNN_F32;
    float dw = 0.f, db = 0.f;
    if (c < w.C)
        for (long long row = static_cast<long long>(blockIdx.y) * 8 + y; row < rows; row += static_cast<long long>(gridDim.y) * 8) {
            if (row % w.S >= count(w.lengths, static_cast<int>(row / w.S), w.S)) continue;
            float r[1], dy[1];
            load<1>(w.r, row * w.C + c, rf, r);
            load<1>(w.y, row * w.C + c, yf, dy);
            dw = fmaf(dy[0], (r[0] - w.stats[2 * row]) * w.stats[2 * row + 1], dw);
            db += dy[0];
        }
    s[0][y][lane] = dw, s[1][y][lane] = db;
    __syncthreads();
    if (y < 2 && c < w.C) {
        float sum = 0.f;
        for (int i = 0; i < 8; ++i) sum += s[y][i][lane];
        w.part[(static_cast<long long>(blockIdx.y) * 2 + y) * w.C + c] = sum;
    }
}

// Which kernel takes a row: threads of a team and vectors of a thread.  (A warp needs no barrier, but 16 vectors to a lane
// leave one CTA to an SM: [32768, 2048] forward 172 us against 130.)
struct Fit {
    int v, team, k;
};
Fit fit(const LnArgs &a) {
    const int v = a.C % 4 == 0 ? 4 : 1, nv = a.C / v;
    if (nv <= 32) return {v, 32, 1};
    if (nv <= 64) return {v, 32, 2};
    if (nv <= 128) return {v, 32, 4};
    if (nv <= 256) return {v, 256, 1};
    if (nv <= 512) return {v, 256, 2};
    if (nv <= 1024) return {v, 256, 4};
    if (nv <= 2048) return {v, 256, 8};
    if (nv <= 8192) return {v, 1024, 8};
    return {v, 1024, 0};
}

template <int V, int TEAM, int K>
void forward(const LnArgs &a, cudaStream_t s) {
    constexpr int TEAMS = cta_of<TEAM>() / TEAM;
    const long long rows = static_cast<long long>(a.N) * a.S;
    ln_forward_kernel<V, TEAM, K><<<static_cast<unsigned>((rows + TEAMS - 1) / TEAMS), cta_of<TEAM>(), 0, s>>>(a);
}
template <int V, int TEAM, int K>
void backward(const LnArgs &a, cudaStream_t s) {
    const size_t smem = TEAM == 32 ? 8 * 2 * static_cast<size_t>(a.C) * sizeof(float) : 0;
    ln_backward_kernel<V, TEAM, K><<<ln_backward_rows(a), cta_of<TEAM>(), smem, s>>>(a);
}
template <int V, bool BACK, int TEAM, int K>
void launch_fit(const LnArgs &a, cudaStream_t s) {
    if constexpr (BACK) backward<V, TEAM, K>(a, s);
    else forward<V, TEAM, K>(a, s);
}
template <int V, bool BACK>
void launch(const LnArgs &a, const Fit &f, cudaStream_t s) {
#define PARARNN_LN(TEAM_, K_) \
    if (f.team == TEAM_ && f.k == K_) return launch_fit<V, BACK, TEAM_, K_>(a, s)
    PARARNN_LN(32, 1);
    PARARNN_LN(32, 2);
    PARARNN_LN(32, 4);
    PARARNN_LN(256, 1);
    PARARNN_LN(256, 2);
    PARARNN_LN(256, 4);
    PARARNN_LN(256, 8);
    PARARNN_LN(1024, 8);
    PARARNN_LN(1024, 0);
#undef PARARNN_LN
}

}  // namespace

// CTAs of the backward pass, each of which leaves a row of sums: three to an SM, as fit it at 2048 channels (fewer do where a
// thread has more vectors, or a warp a row), two and one for the widest; fewer where there are fewer rows, and further waves
// where a team would otherwise add up more than 128 rows in one chain, which loses digits (444 CTAs on 2^20 rows: 370 half
// steps of dbias).
int ln_backward_rows(const LnArgs &a) {
    const Fit f = fit(a);
    const long long teams = f.team == 32 ? 8 : 1, groups = (static_cast<long long>(a.N) * a.S + teams - 1) / teams;
    const long long wave = 148 * (f.team > 256 ? 1 : f.k > 4 ? 2 : 3);
    const long long waves = f.k == 0 ? 1 : (groups + 128 * wave - 1) / (128 * wave);
    return static_cast<int>(std::min(groups, wave * waves));
}

cudaError_t launch_ln_forward(const LnArgs &a, cudaStream_t s) {
    const Fit f = fit(a);
    if (f.v == 4) launch<4, false>(a, f, s);
    else launch<1, false>(a, f, s);
    return cudaGetLastError();
}

cudaError_t launch_ln_backward(const LnArgs &a, cudaStream_t s) {
    const Fit f = fit(a);
    if (f.v == 4) launch<4, true>(a, f, s);
    else launch<1, true>(a, f, s);
    cudaError_t e = cudaGetLastError();
    const int rows = ln_backward_rows(a);
    if (e == cudaSuccess && f.k == 0) {
        ln_columns_kernel<<<dim3((a.C + 31) / 32, rows), 256, 0, s>>>(a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
    return launch_rows_sum({a.part, rows, 2ll * a.C, {a.dweight, a.dbias, nullptr}, {a.C, a.C, 0}}, s);
}

}  // namespace pararnn
