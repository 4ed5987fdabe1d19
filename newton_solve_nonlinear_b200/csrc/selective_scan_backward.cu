// selective_scan_backward.cu -- the backward pass of the selective scan (sm_100a).  Formulas: selective_scan.cuh.
#include "rows.cuh"
#include "selective_scan.cuh"

namespace pararnn {
using namespace ss;
namespace {

constexpr int kThr = 128;
constexpr int kK = kSsKeep;  // tokens whose states are formed again at a time

template <int S, int L>
struct Smem {
    static constexpr int CH = 2 * kThr / L, NP = S * L, ROWS = kThr / L;
    static constexpr int ES = CH + (L < 16 ? 32 / L : 2);      // a row of the sums over states, off the banks of the next
    static constexpr int TS = ROWS * NP + (NP < 32 ? NP : 0);  // a token's sums over channels, likewise
    float4 du[kK][CH / 2];  // s and s x of two channels
    float2 v[kK][CH / 2];
    float b[kK][NP], c[kK][NP];
    float e[3][kK][L][ES];        // parts of sum G b, sum a P h and sum c h, summed over L
    float pb[kK][TS], pc[kK][TS];  // parts of db and dc, [ROWS][NP], summed over the rows
};

// One CTA: 2 kThr / L channels of one group, one segment of one sequence, backward in time.  A thread holds S states of
// each of two channels: what it sums over its channels (for db, dc) and over its states (for dx, ds and the inner y)
// leaves 1 / 2 and 1 / S of the values to pass through shared memory, whose bytes are what bounds this kernel next to its
// arithmetic.  Eight tokens at a time: from the kept state their decays and states are formed again into registers, then
// walked backward.  VEC: pairs of channels, and quads of b and c, lie on their own alignment.
template <typename T, int S, int L, bool VEC>
__global__ void __launch_bounds__(kThr, S == 2 ? 3 : 2) ss_backward_kernel(const SsArgs w) {
    using SM = Smem<S, L>;
    constexpr int CH = SM::CH, NP = SM::NP, Q = S / 2;
    constexpr int LT = kThr / (CH / 2), PER = (kK + LT - 1) / LT;
    extern __shared__ __align__(16) char smem[];
    SM &sm = *reinterpret_cast<SM *>(smem);

    const int tid = threadIdx.x, per = w.D / w.G;
    const int tiles = (per + CH - 1) / CH, blocks = tiles * w.G;
    const int tile = blockIdx.x % blocks % tiles, g = blockIdx.x % blocks / tiles;
    const int seg = blockIdx.x / blocks % w.n_seg, b = blockIdx.x / blocks / w.n_seg;
    const int len = row_count(w.lengths, b, w.T);
    const int t_first = seg * w.seg, t_end = min(w.T, t_first + w.seg), t_len = min(t_end, len);
    const long long all = static_cast<long long>(w.B) * w.D * w.N;
    const bool vec = w.N % S == 0, gated = w.gate.p != nullptr;

    // as owner of the states of two channels
    const int pair = tid / L, n0 = tid % L * S, d = g * per + tile * CH + 2 * pair;
    const int owns = min(2, max(0, per - tile * CH - 2 * pair));
    const long long state_at = (static_cast<long long>(b) * w.D + d) * w.N;
    u64 p[2][Q] = {}, da[2][Q] = {};
    float a[2][S] = {};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        if (q >= owns) continue;
#pragma unroll
        for (int i = 0; i < S; ++i)
            if (n0 + i < w.N) a[q][i] = w.a[(static_cast<long long>(d) + q) * w.N + n0 + i] * kLog2eF;
        const float *from = w.n_seg > 1 ? w.rev_state + seg * all : w.dh;
        if (from != nullptr) load_states(p[q], from + state_at + q * w.N, n0, w.N, vec);
    }
    // as the one who prepares and finishes tokens lt + i LT of the channels lc and lc + 1
    const int lc = tid % (CH / 2) * 2, lt = tid / (CH / 2), ld = g * per + tile * CH + lc;
    const int have = min(2, max(0, per - tile * CH - lc));
    float bias[2] = {}, skip[2] = {}, dskip[2] = {}, dbias[2] = {};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        if (q < have && w.dt_bias != nullptr) bias[q] = w.dt_bias[ld + q];
        if (q < have && w.skip != nullptr) skip[q] = w.skip[ld + q];
    }
    const int n_chunk = (max(t_len - t_first, 0) + kK - 1) / kK;
    const int t_start = t_first + max(n_chunk - 1, 0) * kK;
    const T *px = static_cast<const T *>(w.x.p) + b * w.x.sb + ld + (t_start + lt) * w.x.st;
    const T *pdt = static_cast<const T *>(w.dt.p) + b * w.dt.sb + ld + (t_start + lt) * w.dt.st;
    const T *pg = static_cast<const T *>(w.gate.p) + b * w.gate.sb + ld + (t_start + lt) * w.gate.st;
    const T *pdy = static_cast<const T *>(w.dy.p) + b * w.dy.sb + ld + (t_start + lt) * w.dy.st;
    constexpr int BW = VEC ? 4 : 1, BROW = NP / BW, NB = (kK * BROW + kThr - 1) / kThr;
    const int bt = tid / BROW, bn = tid % BROW * BW;
    const T *pb = static_cast<const T *>(w.b.p) + b * w.b.sb + g * w.b.sg + (t_start + bt) * w.b.st + bn;
    const T *pc = static_cast<const T *>(w.c.p) + b * w.c.sb + g * w.c.sg + (t_start + bt) * w.c.st + bn;
    const float *pk_at = w.kept + ((static_cast<long long>(b) * ((w.T + kK - 1) / kK) + t_start / kK) * w.D + d) * w.N;

    Raw<T> nx[PER], nt[PER], ng[PER], ny[PER], cx[PER], cg[PER], cy[PER];  // the next tokens' elements, and the present ones'
    RawN<T, BW> nb[NB], nc[NB];
    float slope[PER][2], sig[PER][2];  // of the softplus; the gate's sigmoid
    u64 hk[2][Q] = {};                 // the next kept states
    auto fetch = [&](int t0) {
        const int left = t_len - t0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = lt + i * LT, n = t < kK && t < left ? have : 0;
            nx[i] = load_raw<VEC>(px + i * LT * w.x.st, n);
            nt[i] = load_raw<VEC>(pdt + i * LT * w.dt.st, n);
            ng[i] = load_raw<VEC>(pg + i * LT * w.gate.st, gated ? n : 0);
            ny[i] = load_raw<VEC>(pdy + i * LT * w.dy.st, n);
        }
        px -= kK * w.x.st, pdt -= kK * w.dt.st, pg -= kK * w.gate.st, pdy -= kK * w.dy.st;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int t = bt + i * (kThr / BROW);
            const bool on = t < kK && t < left && bn < w.N;
            nb[i] = load_n<BW>(pb + i * (kThr / BROW) * w.b.st, on);
            nc[i] = load_n<BW>(pc + i * (kThr / BROW) * w.c.st, on);
        }
        pb -= kK * w.b.st, pc -= kK * w.c.st;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (q < owns) load_states(hk[q], pk_at + q * w.N, n0, w.N, vec);
        pk_at -= static_cast<long long>(w.D) * w.N;
    };
    auto stage = [&](int t0) {
        float s[PER][2], v[PER][2];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            upk(value(nt[i]), s[i][0], s[i][1]), upk(value(ny[i]), v[i][0], v[i][1]);
            s[i][0] += bias[0], s[i][1] += bias[1];
            slope[i][0] = slope[i][1] = 1.f;
        }
        if (w.softplus) {
#pragma unroll
            for (int i = 0; i < PER; ++i) s[i][0] = softplus(s[i][0], slope[i][0]), s[i][1] = softplus(s[i][1], slope[i][1]);
        }
        if (gated) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                float z[2];
                upk(value(ng[i]), z[0], z[1]);
#pragma unroll
                for (int q = 0; q < 2; ++q) sig[i][q] = sigmoid_of(z[q]), v[i][q] *= z[q] * sig[i][q];
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = lt + i * LT;
            const bool on = t0 + t < t_len;
            float x[2];
            upk(value(nx[i]), x[0], x[1]);
            s[i][0] = on ? s[i][0] : 0.f, s[i][1] = on ? s[i][1] : 0.f;
            if (t < kK) {
                sm.du[t][lc / 2] = make_float4(s[i][0], s[i][1], s[i][0] * x[0], s[i][1] * x[1]);
                sm.v[t][lc / 2] = make_float2(v[i][0], v[i][1]);
            }
            cx[i] = nx[i], cg[i] = ng[i], cy[i] = ny[i];
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int t = bt + i * (kThr / BROW);
            if (t < kK) store_n(&sm.b[t][bn], nb[i]), store_n(&sm.c[t][bn], nc[i]);
        }
    };

    if (n_chunk > 0) {
        fetch(t_start);
        stage(t_start);
    }
    for (int k = n_chunk - 1, t0 = t_start; k >= 0; --k, t0 -= kK) {
        __syncthreads();
        u64 first[2][Q], h[kK][2][Q], e[kK][2][Q];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < Q; ++i) first[q][i] = hk[q][i];
        if (k > 0) fetch(t0 - kK);
#pragma unroll
        for (int t = 0; t < kK; ++t) {
            const float4 du = sm.du[t][pair];
            u64 bb[Q];
            load_pairs(bb, &sm.b[t][n0]);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float st = q == 0 ? du.x : du.y, u = q == 0 ? du.z : du.w;
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    const u64 before = t == 0 ? first[q][i] : h[t == 0 ? 0 : t - 1][q][i];
                    float b0, b1, h0, h1;
                    upk(bb[i], b0, b1), upk(before, h0, h1);
                    e[t][q][i] = decay_less_one(pk(st * a[q][2 * i], st * a[q][2 * i + 1]));
                    h[t][q][i] = fma2(e[t][q][i], before, pk(fmaf(u, b0, h0), fmaf(u, b1, h1)));
                }
            }
        }
#pragma unroll
        for (int t = kK - 1; t >= 0; --t) {
            const float4 du = sm.du[t][pair];
            const float2 vv = sm.v[t][pair];
            u64 bb[Q], cc[Q], db[Q], dc[Q];
            load_pairs(bb, &sm.b[t][n0]);
            load_pairs(cc, &sm.c[t][n0]);
            float e1[2], e2[2], e3[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float st = q == 0 ? du.x : du.y, u = q == 0 ? du.z : du.w, v = q == 0 ? vv.x : vv.y;
                u64 x1 = 0, x2 = 0, x3 = 0;
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    const u64 before = t == 0 ? first[q][i] : h[t == 0 ? 0 : t - 1][q][i];
                    float c0, c1, p0, p1, h0, h1, g0, g1, m0, m1, d0, d1;
                    upk(cc[i], c0, c1), upk(p[q][i], p0, p1), upk(h[t][q][i], h0, h1);
                    g0 = fmaf(v, c0, p0), g1 = fmaf(v, c1, p1);
                    const u64 G = pk(g0, g1);
                    if (q == 0) {
                        dc[i] = pk(v * h0, v * h1), db[i] = pk(u * g0, u * g1);
                    } else {
                        upk(dc[i], d0, d1);
                        dc[i] = pk(fmaf(v, h0, d0), fmaf(v, h1, d1));
                        upk(db[i], d0, d1);
                        db[i] = pk(fmaf(u, g0, d0), fmaf(u, g1, d1));
                    }
                    x1 = i == 0 ? mul2(G, bb[i]) : fma2(G, bb[i], x1);
                    p[q][i] = fma2(e[t][q][i], G, G);
                    const u64 m = mul2(p[q][i], before), aa = pk(a[q][2 * i], a[q][2 * i + 1]);
                    x2 = i == 0 ? mul2(m, aa) : fma2(m, aa, x2);
                    upk(m, m0, m1), upk(da[q][i], d0, d1);
                    da[q][i] = pk(fmaf(st, m0, d0), fmaf(st, m1, d1));
                    if (gated) x3 = i == 0 ? mul2(cc[i], h[t][q][i]) : fma2(cc[i], h[t][q][i], x3);
                }
                e1[q] = pair_sum(x1), e2[q] = pair_sum(x2), e3[q] = pair_sum(x3);
            }
            *reinterpret_cast<float2 *>(&sm.e[0][t][tid % L][2 * pair]) = make_float2(e1[0], e1[1]);
            *reinterpret_cast<float2 *>(&sm.e[1][t][tid % L][2 * pair]) = make_float2(e2[0], e2[1]);
            if (gated) *reinterpret_cast<float2 *>(&sm.e[2][t][tid % L][2 * pair]) = make_float2(e3[0], e3[1]);
            store_pairs(&sm.pb[t][pair * NP + n0], db);
            store_pairs(&sm.pc[t][pair * NP + n0], dc);
        }
        __syncthreads();
        // the sums over the states: dx, ddt, dgate
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = lt + i * LT, n = t < kK && t0 + t < t_len ? have : 0;
            if (n == 0) continue;
            float e1[2] = {}, e2[2] = {}, e3[2] = {}, x[2], z[2], y[2], ddt[2], dx[2], dg[2];
#pragma unroll
            for (int l = 0; l < L; ++l) {
                const float2 q1 = *reinterpret_cast<const float2 *>(&sm.e[0][t][l][lc]);
                const float2 q2 = *reinterpret_cast<const float2 *>(&sm.e[1][t][l][lc]);
                e1[0] += q1.x, e1[1] += q1.y, e2[0] += q2.x, e2[1] += q2.y;
                if (gated) {
                    const float2 q3 = *reinterpret_cast<const float2 *>(&sm.e[2][t][l][lc]);
                    e3[0] += q3.x, e3[1] += q3.y;
                }
            }
            upk(value(cx[i]), x[0], x[1]), upk(value(cg[i]), z[0], z[1]), upk(value(cy[i]), y[0], y[1]);
            const float4 du = sm.du[t][lc / 2];
            const float2 vv = sm.v[t][lc / 2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float v = q == 0 ? vv.x : vv.y;
                ddt[q] = fmaf(x[q], e1[q], e2[q] * 0.693147181f) * slope[i][q];
                dx[q] = fmaf(skip[q], v, (q == 0 ? du.x : du.y) * e1[q]);
                dskip[q] = fmaf(v, x[q], dskip[q]);
                dbias[q] += ddt[q];
                if (gated) dg[q] = y[q] * fmaf(skip[q], x[q], e3[q]) * sig[i][q] * fmaf(z[q], 1.f - sig[i][q], 1.f);
            }
            const long long to = (static_cast<long long>(b) * w.T + t0 + t) * w.D + ld;
            store_pair<VEC>(static_cast<T *>(w.dx) + to, pk(dx[0], dx[1]), n);
            store_pair<VEC>(static_cast<T *>(w.ddt) + to, pk(ddt[0], ddt[1]), n);
            if (gated) store_pair<VEC>(static_cast<T *>(w.dgate) + to, pk(dg[0], dg[1]), n);
        }
        // the sums over the CTA's channels: its part of db and dc
#pragma unroll
        for (int o = tid; o < kK * NP; o += kThr) {
            const int t = o / NP, n = o % NP;
            if (n < w.N && t0 + t < t_len) {
                float sb = 0.f, sc = 0.f;
#pragma unroll
                for (int r = 0; r < SM::ROWS; ++r) sb += sm.pb[t][r * NP + n], sc += sm.pc[t][r * NP + n];
                const long long to = (((static_cast<long long>(tile) * w.B + b) * w.T + t0 + t) * w.G + g) * w.N + n;
                w.part_b[to] = sb;
                w.part_c[to] = sc;
            }
        }
        if (k > 0) {
            __syncthreads();  // du and v of this chunk have been read
            stage(t0 - kK);
        }
    }
    {  // nothing stands behind a sequence
        const long long out = static_cast<long long>(b) * w.T * w.D + ld;
        for (int t = max(t_len, t_first) + lt; t < t_end; t += LT) {
            const long long to = out + static_cast<long long>(t) * w.D;
            store_pair<VEC>(static_cast<T *>(w.dx) + to, 0ull, have);
            store_pair<VEC>(static_cast<T *>(w.ddt) + to, 0ull, have);
            if (gated) store_pair<VEC>(static_cast<T *>(w.dgate) + to, 0ull, have);
        }
    }
    // a row of the parameters' sums: da, dskip, ddt_bias
    float *part = w.part_a + (static_cast<long long>(seg) * w.B + b) * w.D * (w.N + 2);
#pragma unroll
    for (int q = 0; q < 2; ++q)
        if (q < owns) {
            store_states(da[q], part + (static_cast<long long>(d) + q) * w.N, n0, w.N, vec && w.D % 2 == 0);
            if (seg == 0 && w.dh0 != nullptr) store_states(p[q], w.dh0 + state_at + q * w.N, n0, w.N, vec);
        }
    __syncthreads();
    float2 *s_sum = reinterpret_cast<float2 *>(smem);
    s_sum[tid] = make_float2(dskip[0], dskip[1]), s_sum[kThr + tid] = make_float2(dbias[0], dbias[1]);
    __syncthreads();
    if (tid < CH / 2) {
        float2 s = make_float2(0.f, 0.f), q = s;
#pragma unroll
        for (int i = 0; i < LT; ++i) {
            const float2 u = s_sum[tid + i * (CH / 2)], v = s_sum[kThr + tid + i * (CH / 2)];
            s.x += u.x, s.y += u.y, q.x += v.x, q.y += v.y;
        }
        float *to = part + static_cast<long long>(w.D) * w.N + ld;
        if (have > 0) to[0] = s.x, to[w.D] = q.x;
        if (have > 1) to[1] = s.y, to[w.D + 1] = q.y;
    }
}

// db, dc = the sums over the tiles of a group; zero behind the sequences
template <typename T>
__global__ void __launch_bounds__(256) ss_tiles_sum_kernel(const SsArgs w, int tiles) {
    const long long n = static_cast<long long>(w.B) * w.T * w.G * w.N, row = static_cast<long long>(w.G) * w.N;
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<long long>(gridDim.x) * 256) {
        const long long bt = i / row;
        const int b = static_cast<int>(bt / w.T), t = static_cast<int>(bt % w.T);
        float sb = 0.f, sc = 0.f;
        if (t < row_count(w.lengths, b, w.T))
            for (int k = 0; k < tiles; ++k) sb += w.part_b[k * n + i], sc += w.part_c[k * n + i];
        static_cast<T *>(w.db)[i] = from_f<T>(sb);
        static_cast<T *>(w.dc)[i] = from_f<T>(sc);
    }
}

template <typename T, int S, int L, bool VEC>
cudaError_t launch(const SsArgs &a, cudaStream_t s) {
    constexpr int bytes = sizeof(Smem<S, L>);
    static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
    const auto kernel = ss_backward_kernel<T, S, L, VEC>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(ss_backward_tiles(a)) * a.G * a.n_seg * a.B, kThr, bytes, s>>>(a);
    return cudaGetLastError();
}
int lanes(int N) { return N <= 4 ? 2 : N <= 8 ? 4 : N <= 16 ? 8 : N <= 32 ? 16 : 32; }
template <typename T, bool VEC>
cudaError_t launch_of(const SsArgs &a, cudaStream_t s) {
    switch (lanes(a.N)) {
        case 2: return launch<T, 2, 2, VEC>(a, s);
        case 4: return launch<T, 2, 4, VEC>(a, s);
        case 8: return launch<T, 2, 8, VEC>(a, s);
        case 16: return launch<T, 2, 16, VEC>(a, s);
        default: return launch<T, 2, 32, VEC>(a, s);
    }
}

}  // namespace

int ss_backward_tiles(const SsArgs &a) {
    const int per = a.D / a.G, ch = 2 * kThr / lanes(a.N);
    return (per + ch - 1) / ch;
}

cudaError_t launch_ss_backward(const SsArgs &a, cudaStream_t s) {
    cudaError_t e = launch_ss_reverse_states(a, s);
    const bool vec = ss_pairs_ok(a);
    if (e == cudaSuccess) {
        if (a.dtype == PARARNN_F32) e = vec ? launch_of<float, true>(a, s) : launch_of<float, false>(a, s);
        else e = vec ? launch_of<__nv_bfloat16, true>(a, s) : launch_of<__nv_bfloat16, false>(a, s);
    }
    const long long n = static_cast<long long>(a.B) * a.T * a.G * a.N, rows = static_cast<long long>(a.n_seg) * a.B;
    const long long dn = static_cast<long long>(a.D) * a.N;
    if (e == cudaSuccess) {
        const unsigned grid = static_cast<unsigned>(n / 256 + 1 < 148 * 8 ? n / 256 + 1 : 148 * 8);
        const int tiles = ss_backward_tiles(a);
        if (a.dtype == PARARNN_F32) ss_tiles_sum_kernel<float><<<grid, 256, 0, s>>>(a, tiles);
        else ss_tiles_sum_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a, tiles);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
    return launch_rows_sum({a.part_a, rows, dn + 2ll * a.D, {a.da, a.dskip, a.ddt_bias}, {dn, a.D, a.D}}, s);
}

}  // namespace pararnn
