// selective_scan_backward.cu -- the backward pass of the selective scan (sm_100a).  Formulas: selective_scan.cuh.
#include "rows.cuh"
#include "selective_scan.cuh"

namespace pararnn {
using namespace ss;
namespace {

constexpr int kThr = 128;
constexpr int kK = kSsKeep;  // tokens whose states are formed again at a time

template <int L>
struct Tile {
    static constexpr int CH = 2 * kThr / L, NP = 4 * L, ROWS = kThr / L;
    static constexpr int ES = CH + 32 / L;                      // a row of the sums over states, off the banks of the next
    static constexpr int TS = ROWS * NP + (NP < 32 ? NP : 0);   // a token's sums over channels
    // floats: s, s, s x, s x and v, v of each token and channel; b and c; sums over states (3); sums over channels (2)
    static constexpr int FLOATS = kK * CH * 6 + 2 * kK * NP + 3 * kK * L * ES + 2 * kK * TS;
};

// One CTA: 256 / L channels of one group, one segment of one sequence, backward in time.  A thread holds two channels and
// four states of each: what it sums over its channels (for db, dc) and over its states (for dx, ds and the inner y) leaves
// half and a quarter of the values for shared memory to sum.  Eight tokens at a time: from the kept state their decays and
// states are formed again into registers, then walked backward.
template <typename T, int L>
__global__ void __launch_bounds__(kThr) ss_backward_kernel(const SsArgs w) {
    using TL = Tile<L>;
    constexpr int CH = TL::CH, NP = TL::NP, PER = kK * CH / kThr, LT = kThr / CH;
    extern __shared__ __align__(16) float smem[];
    float4 *s_du = reinterpret_cast<float4 *>(smem);                   // [kK][CH]
    float2 *s_v = reinterpret_cast<float2 *>(smem + kK * CH * 4);      // [kK][CH]
    float *s_b = smem + kK * CH * 6, *s_c = s_b + kK * NP;             // [kK][NP]
    float *s_e = s_c + kK * NP;                                        // [3][kK][L][ES]
    float *s_pb = s_e + 3 * kK * L * TL::ES, *s_pc = s_pb + kK * TL::TS;  // [kK][ROWS][NP]

    const int tid = threadIdx.x, per = w.D / w.G;
    const int tiles = (per + CH - 1) / CH, blocks = tiles * w.G;
    const int tile = blockIdx.x % blocks % tiles, g = blockIdx.x % blocks / tiles;
    const int seg = blockIdx.x / blocks % w.n_seg, b = blockIdx.x / blocks / w.n_seg;
    const int len = row_count(w.lengths, b, w.T);
    const int t_first = seg * w.seg, t_end = min(w.T, t_first + w.seg), t_len = min(t_end, len);
    const long long all = static_cast<long long>(w.B) * w.D * w.N;
    const int groups = (w.T + kK - 1) / kK;
    const bool vec = w.N % 4 == 0, gated = w.gate.p != nullptr;

    // as owner of the states of two channels
    const int row = tid / L, n0 = tid % L * 4, c0 = 2 * row;
    u64 a[2][2] = {}, p[2][2] = {}, da[2][2] = {};
    bool owner[2];
    long long state_at[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int c = tile * CH + c0 + q, d = g * per + c;
        owner[q] = c < per;
        state_at[q] = (static_cast<long long>(b) * w.D + d) * w.N;
        if (owner[q]) {
            load_states(a[q], w.a + static_cast<long long>(d) * w.N, n0, w.N, false);
#pragma unroll
            for (int i = 0; i < 2; ++i) a[q][i] = mul2(a[q][i], splat(kLog2eF));
            const float *from = w.n_seg > 1 ? w.rev_state + seg * all : w.dh;
            if (from != nullptr) load_states(p[q], from + state_at[q], n0, w.N, false);
        }
    }
    // as the one who prepares and finishes tokens lt + i LT of channel lch
    const int lch = tid % CH, lt = tid / CH, ld = g * per + tile * CH + lch;
    const bool loads = tile * CH + lch < per;
    const float bias = loads && w.dt_bias != nullptr ? w.dt_bias[ld] : 0.f;
    const float skip = loads && w.skip != nullptr ? w.skip[ld] : 0.f;
    const T *px = static_cast<const T *>(w.x.p) + b * w.x.sb + ld;
    const T *pdt = static_cast<const T *>(w.dt.p) + b * w.dt.sb + ld;
    const T *pg = static_cast<const T *>(w.gate.p) + b * w.gate.sb + ld;
    const T *pdy = static_cast<const T *>(w.dy.p) + b * w.dy.sb + ld;
    const T *pb = static_cast<const T *>(w.b.p) + b * w.b.sb + g * w.b.sg;
    const T *pc = static_cast<const T *>(w.c.p) + b * w.c.sb + g * w.c.sg;
    constexpr int NB = (kK * NP + kThr - 1) / kThr;

    float nx[PER], nt[PER], ng[PER], ny[PER], nb[NB], nc[NB];  // the next tokens, as they are
    float cx[PER], cr[PER], cg[PER], cy[PER];                  // the present ones: x, raw step, gate, dy
    u64 hk[2][2] = {};                                         // the next kept states
    float dskip = 0.f, dbias = 0.f;
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = t0 + lt + i * LT;
            const bool on = loads && t < t_len;
            nx[i] = on ? to_f(px[t * w.x.st]) : 0.f;
            nt[i] = on ? to_f(pdt[t * w.dt.st]) : 0.f;
            ny[i] = on ? to_f(pdy[t * w.dy.st]) : 0.f;
            ng[i] = on && gated ? to_f(pg[t * w.gate.st]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int e = tid + i * kThr, t = t0 + e / NP, n = e % NP;
            const bool on = e < kK * NP && n < w.N && t < t_len;
            nb[i] = on ? to_f(pb[t * w.b.st + n]) : 0.f;
            nc[i] = on ? to_f(pc[t * w.c.st + n]) : 0.f;
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (owner[q])
                load_states(hk[q], w.kept + ((static_cast<long long>(b) * groups + t0 / kK) * w.D + g * per + tile * CH + c0 + q) * w.N,
                            n0, w.N, vec);
    };
    auto stage = [&](int t0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = lt + i * LT;
            float s = 0.f, v = 0.f;
            cx[i] = nx[i], cg[i] = ng[i], cy[i] = ny[i], cr[i] = nt[i] + bias;
            if (loads && t0 + t < t_len) {
                s = w.softplus ? softplus(cr[i]) : cr[i];
                v = gated ? gate_with(ny[i], ng[i]) : ny[i];
            }
            const float u = s * nx[i];
            s_du[t * CH + lch] = make_float4(s, s, u, u);
            s_v[t * CH + lch] = make_float2(v, v);
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int e = tid + i * kThr;
            if (e < kK * NP) s_b[e] = nb[i], s_c[e] = nc[i];
        }
    };

    const int n_chunk = (max(t_len - t_first, 0) + kK - 1) / kK;
    if (n_chunk > 0) {
        fetch(t_first + (n_chunk - 1) * kK);
        stage(t_first + (n_chunk - 1) * kK);
    }
    for (int k = n_chunk - 1; k >= 0; --k) {
        const int t0 = t_first + k * kK;
        __syncthreads();
        u64 first[2][2], h[kK][2][2], e[kK][2][2];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 2; ++i) first[q][i] = hk[q][i];
        if (k > 0) fetch(t0 - kK);
#pragma unroll
        for (int t = 0; t < kK; ++t) {
            u64 bb[2];
            load_pairs(bb, s_b + t * NP + n0);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const ulonglong2 du = *reinterpret_cast<const ulonglong2 *>(s_du + t * CH + c0 + q);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const u64 before = t == 0 ? first[q][i] : h[t == 0 ? 0 : t - 1][q][i];
                    e[t][q][i] = decay_less_one(mul2(du.x, a[q][i]));
                    h[t][q][i] = fma2(e[t][q][i], before, fma2(du.y, bb[i], before));
                }
            }
        }
#pragma unroll
        for (int t = kK - 1; t >= 0; --t) {
            u64 bb[2], cc[2], db[2] = {0, 0}, dc[2] = {0, 0};
            load_pairs(bb, s_b + t * NP + n0);
            load_pairs(cc, s_c + t * NP + n0);
            float e1[2], e2[2], e3[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const ulonglong2 du = *reinterpret_cast<const ulonglong2 *>(s_du + t * CH + c0 + q);
                const u64 v = *reinterpret_cast<const u64 *>(s_v + t * CH + c0 + q);
                u64 x1 = 0, x2 = 0, x3 = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const u64 before = t == 0 ? first[q][i] : h[t == 0 ? 0 : t - 1][q][i];
                    const u64 G = fma2(v, cc[i], p[q][i]);
                    dc[i] = fma2(v, h[t][q][i], dc[i]);
                    db[i] = fma2(G, du.y, db[i]);
                    x1 = fma2(G, bb[i], x1);
                    p[q][i] = fma2(e[t][q][i], G, G);
                    const u64 m = mul2(p[q][i], before);
                    x2 = fma2(m, a[q][i], x2);
                    da[q][i] = fma2(m, du.x, da[q][i]);
                    x3 = fma2(cc[i], h[t][q][i], x3);
                }
                e1[q] = pair_sum(x1), e2[q] = pair_sum(x2), e3[q] = pair_sum(x3);
            }
            const int at = (t * L + tid % L) * TL::ES + c0;
            *reinterpret_cast<float2 *>(s_e + at) = make_float2(e1[0], e1[1]);
            *reinterpret_cast<float2 *>(s_e + kK * L * TL::ES + at) = make_float2(e2[0], e2[1]);
            if (gated) *reinterpret_cast<float2 *>(s_e + 2 * kK * L * TL::ES + at) = make_float2(e3[0], e3[1]);
            *reinterpret_cast<ulonglong2 *>(s_pb + t * TL::TS + row * NP + n0) = make_ulonglong2(db[0], db[1]);
            *reinterpret_cast<ulonglong2 *>(s_pc + t * TL::TS + row * NP + n0) = make_ulonglong2(dc[0], dc[1]);
        }
        __syncthreads();
        // the sums over the states: dx, ddt, dgate
        const long long out = (static_cast<long long>(b) * w.T + t0) * w.D + ld;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = lt + i * LT;
            float e1 = 0.f, e2 = 0.f, e3 = 0.f;
#pragma unroll
            for (int l = 0; l < L; ++l) {
                const int at = (t * L + l) * TL::ES + lch;
                e1 += s_e[at], e2 += s_e[kK * L * TL::ES + at];
                if (gated) e3 += s_e[2 * kK * L * TL::ES + at];
            }
            if (!loads || t0 + t >= t_len) continue;
            const float4 du = s_du[t * CH + lch];
            const float v = s_v[t * CH + lch].x;
            float ds = fmaf(cx[i], e1, e2 * 0.693147181f);
            if (w.softplus) ds *= sigmoid_of(cr[i]);
            const long long to = out + static_cast<long long>(t) * w.D;
            static_cast<T *>(w.dx)[to] = from_f<T>(fmaf(skip, v, du.x * e1));
            static_cast<T *>(w.ddt)[to] = from_f<T>(ds);
            dskip = fmaf(v, cx[i], dskip);
            dbias += ds;
            if (gated) {
                const float z = sigmoid_of(cg[i]), y = fmaf(skip, cx[i], e3);
                static_cast<T *>(w.dgate)[to] = from_f<T>(cy[i] * y * z * fmaf(cg[i], 1.f - z, 1.f));
            }
        }
        // the sums over the CTA's channels: its part of db and dc
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int o = tid + i * kThr, t = o / NP, n = o % NP;
            if (o < kK * NP && n < w.N && t0 + t < t_len) {
                float sb = 0.f, sc = 0.f;
#pragma unroll 8
                for (int r = 0; r < TL::ROWS; ++r) {
                    sb += s_pb[t * TL::TS + r * NP + n];
                    sc += s_pc[t * TL::TS + r * NP + n];
                }
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
    if (loads) {  // nothing stands behind a sequence
        const long long out = static_cast<long long>(b) * w.T * w.D + ld;
        for (int t = max(t_len, t_first) + lt; t < t_end; t += LT) {
            const long long to = out + static_cast<long long>(t) * w.D;
            static_cast<T *>(w.dx)[to] = from_f<T>(0.f);
            static_cast<T *>(w.ddt)[to] = from_f<T>(0.f);
            if (gated) static_cast<T *>(w.dgate)[to] = from_f<T>(0.f);
        }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q)
        if (owner[q]) {
            store_states(da[q], w.part_a + seg * all + state_at[q], n0, w.N, false);
            if (seg == 0 && w.dh0 != nullptr) store_states(p[q], w.dh0 + state_at[q], n0, w.N, false);
        }
    __syncthreads();
    smem[tid] = dskip, smem[kThr + tid] = dbias;
    __syncthreads();
    if (tid < CH && loads) {
        float s = 0.f, q = 0.f;
#pragma unroll
        for (int i = 0; i < LT; ++i) s += smem[tid + i * CH], q += smem[kThr + tid + i * CH];
        const long long to = (static_cast<long long>(seg) * w.B + b) * w.D + ld;
        w.part_skip[to] = s;
        w.part_bias[to] = q;
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

template <typename T, int L>
cudaError_t launch(const SsArgs &a, cudaStream_t s) {
    constexpr int bytes = Tile<L>::FLOATS * 4;
    static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
    const cudaError_t e = cudaFuncSetAttribute(ss_backward_kernel<T, L>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(ss_backward_tiles(a)) * a.G * a.n_seg * a.B;
    ss_backward_kernel<T, L><<<grid, kThr, bytes, s>>>(a);
    return cudaGetLastError();
}
int lanes(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }
template <typename T>
cudaError_t launch_of(const SsArgs &a, cudaStream_t s) {
    switch (lanes(a.N)) {
        case 2: return launch<T, 2>(a, s);
        case 4: return launch<T, 4>(a, s);
        case 8: return launch<T, 8>(a, s);
        default: return launch<T, 16>(a, s);
    }
}
}  // namespace

int ss_backward_tiles(const SsArgs &a) {
    const int per = a.D / a.G, ch = 2 * kThr / lanes(a.N);
    return (per + ch - 1) / ch;
}

cudaError_t launch_ss_backward(const SsArgs &a, cudaStream_t s) {
    cudaError_t e = launch_ss_reverse_states(a, s);
    if (e == cudaSuccess) e = a.dtype == PARARNN_F32 ? launch_of<float>(a, s) : launch_of<__nv_bfloat16>(a, s);
    const long long n = static_cast<long long>(a.B) * a.T * a.G * a.N, rows = static_cast<long long>(a.n_seg) * a.B;
    const long long dn = static_cast<long long>(a.D) * a.N;
    if (e == cudaSuccess) {
        const unsigned grid = static_cast<unsigned>(n / 256 + 1 < 148 * 8 ? n / 256 + 1 : 148 * 8);
        const int tiles = ss_backward_tiles(a);
        if (a.dtype == PARARNN_F32) ss_tiles_sum_kernel<float><<<grid, 256, 0, s>>>(a, tiles);
        else ss_tiles_sum_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a, tiles);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) e = launch_rows_sum(a.part_a, a.da, rows, dn, dn, s);
    if (e == cudaSuccess) e = launch_rows_sum(a.part_skip, a.dskip, rows, a.D, a.D, s);
    if (e == cudaSuccess) e = launch_rows_sum(a.part_bias, a.ddt_bias, rows, a.D, a.D, s);
    return e;
}

}  // namespace pararnn
