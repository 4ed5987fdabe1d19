// selective_scan_backward.cu -- the backward pass of the selective scan (sm_100a).  Formulas: selective_scan.cuh.
#include "rows.cuh"
#include "selective_scan.cuh"

namespace pararnn {
using namespace ss;
namespace {

constexpr int kThr = 128;    // threads that hold states; as many again prepare and finish tokens
constexpr int kK = kSsKeep;  // tokens whose states are formed again at a time

template <int S, int L>
struct Smem {  // two of each, for groups of kK tokens in turn
    static constexpr int CH = 2 * kThr / L, NP = S * L, ROWS = kThr / L;
    static constexpr int ES = CH + (L < 16 ? 32 / L : 2);      // a row of the sums over states, off the banks of the next
    static constexpr int TS = ROWS * NP + (NP < 32 ? NP : 0);  // a token's sums over channels, likewise
    float4 du[2][kK][CH / 2];  // s and s x of two channels
    float2 v[2][kK][CH / 2];
    float b[2][kK][NP], c[2][kK][NP];
    float e[2][3][kK][L][ES];            // parts of sum G b, sum a P h and sum c h, summed over L
    float pb[2][kK][TS], pc[2][kK][TS];  // parts of db and dc, [ROWS][NP], summed over the rows
    float4 sums[kThr];                   // dskip and ddt_bias of each finishing thread's two channels
};

// all threads of the CTA, which come from different places of the code
__device__ __forceinline__ void meet() { asm volatile("bar.sync 1, %0;" ::"n"(2 * kThr) : "memory"); }

// A launch has 128 registers to a thread.  The threads that hold states take more, the others make do with the rest: the two
// together are what was there.  The others hold more in fp32, and spill with fewer (training step of 4 x 4096 x 2048 x 16 in
// bf16: 1777 us with 168 to the states' threads, 1523 with 160, 1540 with 152; 4 x 2048 x 2048 x 16 in fp32: 1152, 1073, 885).
constexpr int kRegs = 128;
template <typename T>
constexpr int kStateRegs = sizeof(T) == 4 ? 152 : 160;
template <typename T>
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStateRegs<T>)); }
template <typename T>
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(2 * kRegs - kStateRegs<T>)); }

// One CTA: 2 kThr / L channels of one group, one segment of one sequence, backward in time, eight tokens at a time.
//   Four warps hold the states: a thread has S of each of two channels.  From the kept state its decays and states are formed
// again into registers, then walked backward.  What it sums over its channels (for db, dc) and over its states (for dx, ds
// and the inner y) leaves 1 / 2 and 1 / S of the values to pass through shared memory.
//   Four more prepare the next eight tokens, and finish the last ones: those sums, the gradients of each token and channel,
// and the CTA's part of db and dc.  4 x 4096 x 2048 x 16 in bf16: 975 us, 40 instructions to a state issued in 62 % of the
// cycles.  (Preparing and finishing in the states' own warps took a fifth longer.)  VEC: pairs of channels, and quads of b and
// c, lie on their own alignment.
template <typename T, int S, int L, bool VEC>
__global__ void __launch_bounds__(2 * kThr, 2) ss_backward_kernel(const SsArgs w) {
    using SM = Smem<S, L>;
    constexpr int CH = SM::CH, NP = SM::NP, Q = S / 2;
    extern __shared__ __align__(16) char smem[];
    SM &sm = *reinterpret_cast<SM *>(smem);

    const int per = w.D / w.G, tiles = (per + CH - 1) / CH, blocks = tiles * w.G;
    const int tile = blockIdx.x % blocks % tiles, g = blockIdx.x % blocks / tiles;
    const int seg = blockIdx.x / blocks % w.n_seg, b = blockIdx.x / blocks / w.n_seg;
    const int len = row_count(w.lengths, b, w.T);
    const int t_first = seg * w.seg, t_end = min(w.T, t_first + w.seg), t_len = min(t_end, len);
    const bool gated = w.gate.p != nullptr;
    const int n_chunk = (max(t_len - t_first, 0) + kK - 1) / kK;
    const int t_start = t_first + max(n_chunk - 1, 0) * kK;
    // a row of the parameters' sums: da, dskip, ddt_bias
    float *part = w.part_a + (static_cast<long long>(seg) * w.B + b) * w.D * (w.N + 2);

    if (threadIdx.x < kThr) {
        take_registers<T>();
        const int tid = threadIdx.x, pair = tid / L, n0 = tid % L * S, d = g * per + tile * CH + 2 * pair;
        const int owns = min(2, max(0, per - tile * CH - 2 * pair));
        const bool vec = w.N % S == 0;
        const long long at_d = (static_cast<long long>(b) * w.D + d) * w.N, all = static_cast<long long>(w.B) * w.D * w.N;
        u64 p[2][Q] = {}, hk[2][Q] = {};         // hk: the next kept states
        u64 sum_a[2][Q] = {}, da[2][Q] = {};     // da, of sums over 64 tokens: one long chain would lose digits
        float a[2][S] = {};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (q >= owns) continue;
#pragma unroll
            for (int i = 0; i < S; ++i)
                if (n0 + i < w.N) a[q][i] = rate_of(w.a[(static_cast<long long>(d) + q) * w.N + n0 + i]);
            const float *from = w.n_seg > 1 ? w.rev_state + seg * all : w.dh;
            if (from != nullptr) load_states(p[q], from + at_d + q * w.N, n0, w.N, vec);
        }
        const long long row = static_cast<long long>(w.D) * w.N;
        const float *kept = w.kept + (static_cast<long long>(b) * ((w.T + kK - 1) / kK) + t_start / kK) * row + static_cast<long long>(d) * w.N;
        auto fetch = [&]() {
            if (owns > 0) load_states(hk[0], kept, n0, w.N, vec);
            if (owns > 1) load_states(hk[1], kept + w.N, n0, w.N, vec);
            kept -= row;
        };
        if (n_chunk > 0) fetch();
        meet();
        for (int k = n_chunk - 1; k >= 0; --k) {
            const auto &du_at = sm.du[k & 1];
            const auto &v_at = sm.v[k & 1];
            const auto &b_at = sm.b[k & 1];
            const auto &c_at = sm.c[k & 1];
            auto &e_at = sm.e[k & 1];
            u64 first[2][Q], h[kK][2][Q], e[kK][2][Q];
            unsigned slow = 0;  // a bit to a state and token: its decay leaves G beside e G
            static_assert(kK * 2 * S <= 32, "bits");
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < Q; ++i) first[q][i] = hk[q][i];
            if (k > 0) fetch();
#pragma unroll
            for (int t = 0; t < kK; ++t) {
                const float4 du = du_at[t][pair];
                u64 bb[Q];
                load_pairs(bb, &b_at[t][n0]);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float st = q == 0 ? du.x : du.y, u = q == 0 ? du.z : du.w;
#pragma unroll
                    for (int i = 0; i < Q; ++i) {
                        const u64 before = t == 0 ? first[q][i] : h[t == 0 ? 0 : t - 1][q][i];
                        const u64 xx = pk(st * a[q][2 * i], st * a[q][2 * i + 1]);
                        float b0, b1, x0, x1;
                        upk(bb[i], b0, b1), upk(xx, x0, x1);
                        if (slow_decay(x0)) slow |= 1u << ((t * 2 + q) * S + 2 * i);
                        if (slow_decay(x1)) slow |= 2u << ((t * 2 + q) * S + 2 * i);
                        e[t][q][i] = decay_factor(xx);
                        h[t][q][i] = fma2(e[t][q][i], before, with_rest(xx, u * b0, u * b1, before));
                    }
                }
            }
#pragma unroll
            for (int t = kK - 1; t >= 0; --t) {
                const float4 du = du_at[t][pair];
                const float2 vv = v_at[t][pair];
                u64 bb[Q], cc[Q], db[Q], dc[Q];
                load_pairs(bb, &b_at[t][n0]);
                load_pairs(cc, &c_at[t][n0]);
                float e1[2], e2[2], e3[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float st = q == 0 ? du.x : du.y, u = q == 0 ? du.z : du.w, v = q == 0 ? vv.x : vv.y;
                    u64 x1 = 0, x2 = 0, x3 = 0;
#pragma unroll
                    for (int i = 0; i < Q; ++i) {
                        const u64 before = t == 0 ? first[q][i] : h[t == 0 ? 0 : t - 1][q][i];
                        float c0, c1, p0, p1, h0, h1, m0, m1, d0, d1;
                        upk(cc[i], c0, c1), upk(p[q][i], p0, p1), upk(h[t][q][i], h0, h1);
                        const float g0 = fmaf(v, c0, p0), g1 = fmaf(v, c1, p1);
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
                        const int bit = (t * 2 + q) * S + 2 * i;
                        upk(mul2(e[t][q][i], G), p0, p1);
                        if (slow & 1u << bit) p0 += g0;
                        if (slow & 2u << bit) p1 += g1;
                        p[q][i] = pk(p0, p1);
                        const u64 m = mul2(p[q][i], before), aa = pk(a[q][2 * i], a[q][2 * i + 1]);
                        x2 = i == 0 ? mul2(m, aa) : fma2(m, aa, x2);
                        upk(m, m0, m1), upk(da[q][i], d0, d1);
                        da[q][i] = pk(fmaf(st, m0, d0), fmaf(st, m1, d1));
                        if (gated) x3 = i == 0 ? mul2(cc[i], h[t][q][i]) : fma2(cc[i], h[t][q][i], x3);
                    }
                    e1[q] = pair_sum(x1), e2[q] = pair_sum(x2), e3[q] = pair_sum(x3);
                }
                *reinterpret_cast<float2 *>(&e_at[0][t][tid % L][2 * pair]) = make_float2(e1[0], e1[1]);
                *reinterpret_cast<float2 *>(&e_at[1][t][tid % L][2 * pair]) = make_float2(e2[0], e2[1]);
                if (gated) *reinterpret_cast<float2 *>(&e_at[2][t][tid % L][2 * pair]) = make_float2(e3[0], e3[1]);
                store_pairs(&sm.pb[k & 1][t][pair * NP + n0], db);
                store_pairs(&sm.pc[k & 1][t][pair * NP + n0], dc);
            }
            if ((k & 7) == 0) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int i = 0; i < Q; ++i) sum_a[q][i] = add2(sum_a[q][i], da[q][i]), da[q][i] = 0;
            }
            meet();
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (q < owns) {
                store_states(sum_a[q], part + (static_cast<long long>(d) + q) * w.N, n0, w.N, false);
                if (seg == 0 && w.dh0 != nullptr) store_states(p[q], w.dh0 + at_d + q * w.N, n0, w.N, vec);
            }
        return;
    }

    // SUB threads to each token of a group of eight and each pair of channels lc and lc + 1: they share the sums over the
    // lanes, of which there are more where there are fewer pairs
    give_registers<T>();
    constexpr int LT = kK, PER = 1, SUB = kThr / (CH / 2) / kK;
    static_assert(SUB >= 1 && CH / 2 * SUB <= 32, "the threads of a token and pair are in one warp");
    const int tid = threadIdx.x - kThr;
    const int lc = tid % (CH / 2) * 2, sub = tid / (CH / 2) % SUB, lt = tid / (CH / 2) / SUB, ld = g * per + tile * CH + lc;
    const int have = min(2, max(0, per - tile * CH - lc));
    float bias[2] = {}, skip[2] = {}, dskip[2] = {}, dbias[2] = {};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        if (q < have && w.dt_bias != nullptr) bias[q] = w.dt_bias[ld + q];
        if (q < have && w.skip != nullptr) skip[q] = w.skip[ld + q];
    }
    const T *px = static_cast<const T *>(w.x.p) + b * w.x.sb + ld + (t_start + lt) * w.x.st;
    const T *pdt = static_cast<const T *>(w.dt.p) + b * w.dt.sb + ld + (t_start + lt) * w.dt.st;
    const T *pg = static_cast<const T *>(w.gate.p) + b * w.gate.sb + ld + (t_start + lt) * w.gate.st;
    const T *pdy = static_cast<const T *>(w.dy.p) + b * w.dy.sb + ld + (t_start + lt) * w.dy.st;
    constexpr int BW = VEC ? 4 : 1, BROW = NP / BW, NB = (kK * BROW + kThr - 1) / kThr;
    const int bt = tid / BROW, bn = tid % BROW * BW;
    const T *pb = static_cast<const T *>(w.b.p) + b * w.b.sb + g * w.b.sg + (t_start + bt) * w.b.st + bn;
    const T *pc = static_cast<const T *>(w.c.p) + b * w.c.sb + g * w.c.sg + (t_start + bt) * w.c.st + bn;

    struct Kept {  // of a token and its two channels from its preparation on
        Raw<T> x, g, y;
        float s[2], v[2], slope[2], sig[2];  // the step, v, the softplus' slope, the gate's sigmoid
    };
    Raw<T> nx[PER], nt[PER], ng[PER], ny[PER];  // the next tokens' elements
    RawN<T, BW> nb[NB], nc[NB];
    Kept now[PER], last[PER];
    auto fetch = [&](int t0) {
        const int left = t_len - t0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = lt + i * LT, n = sub == 0 && t < left ? have : 0;
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
    };
    auto stage = [&](int t0, int to) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            last[i] = now[i];
            Kept &n = now[i];
            n.x = nx[i], n.g = ng[i], n.y = ny[i];
            upk(value(nt[i]), n.s[0], n.s[1]), upk(value(ny[i]), n.v[0], n.v[1]);
            n.s[0] += bias[0], n.s[1] += bias[1];
            n.slope[0] = n.slope[1] = 1.f;
        }
        if (w.softplus) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
#pragma unroll
                for (int q = 0; q < 2; ++q) now[i].s[q] = softplus(now[i].s[q], now[i].slope[q]);
        }
        if (gated) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                float z[2];
                upk(value(ng[i]), z[0], z[1]);
#pragma unroll
                for (int q = 0; q < 2; ++q) now[i].sig[q] = sigmoid_of(z[q]), now[i].v[q] *= z[q] * now[i].sig[q];
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = lt + i * LT;
            Kept &n = now[i];
            const bool on = t0 + t < t_len;
            float x[2];
            upk(value(nx[i]), x[0], x[1]);
            n.s[0] = on ? n.s[0] : 0.f, n.s[1] = on ? n.s[1] : 0.f;
            if (sub == 0) {
                sm.du[to][t][lc / 2] = make_float4(n.s[0], n.s[1], n.s[0] * x[0], n.s[1] * x[1]);
                sm.v[to][t][lc / 2] = make_float2(n.v[0], n.v[1]);
            }
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int t = bt + i * (kThr / BROW);
            if (t < kK) store_n(&sm.b[to][t][bn], nb[i]), store_n(&sm.c[to][t][bn], nc[i]);
        }
    };
    auto finish = [&](int t0, int from, const Kept (&of)[PER]) {
        const auto &e_at = sm.e[from];
        // the sums over the states: dx, ddt, dgate
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = lt + i * LT, n = sub == 0 && t0 + t < t_len ? have : 0;
            float e1[2] = {}, e2[2] = {}, e3[2] = {}, x[2], z[2], y[2], ddt[2], dx[2], dg[2];
#pragma unroll
            for (int l0 = 0; l0 < L / SUB; ++l0) {
                const int l = sub * (L / SUB) + l0;
                const float2 q1 = *reinterpret_cast<const float2 *>(&e_at[0][t][l][lc]);
                const float2 q2 = *reinterpret_cast<const float2 *>(&e_at[1][t][l][lc]);
                e1[0] += q1.x, e1[1] += q1.y, e2[0] += q2.x, e2[1] += q2.y;
            }
            if (gated) {
#pragma unroll
                for (int l0 = 0; l0 < L / SUB; ++l0) {
                    const float2 q3 = *reinterpret_cast<const float2 *>(&e_at[2][t][sub * (L / SUB) + l0][lc]);
                    e3[0] += q3.x, e3[1] += q3.y;
                }
            }
#pragma unroll
            for (int o = CH / 2; o < CH / 2 * SUB; o *= 2)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    e1[q] += __shfl_xor_sync(0xffffffffu, e1[q], o);
                    e2[q] += __shfl_xor_sync(0xffffffffu, e2[q], o);
                    e3[q] += __shfl_xor_sync(0xffffffffu, e3[q], o);
                }
            if (n == 0) continue;
            const Kept &o = of[i];
            upk(value(o.x), x[0], x[1]), upk(value(o.g), z[0], z[1]), upk(value(o.y), y[0], y[1]);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                ddt[q] = fmaf(x[q], e1[q], e2[q] * 0.693147181f) * o.slope[q];
                dx[q] = fmaf(skip[q], o.v[q], o.s[q] * e1[q]);
                dskip[q] = fmaf(o.v[q], x[q], dskip[q]);
                dbias[q] += ddt[q];
                if (gated) dg[q] = y[q] * fmaf(skip[q], x[q], e3[q]) * o.sig[q] * fmaf(z[q], 1.f - o.sig[q], 1.f);
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
                for (int r = 0; r < SM::ROWS; ++r) sb += sm.pb[from][t][r * NP + n], sc += sm.pc[from][t][r * NP + n];
                const long long to = (((static_cast<long long>(tile) * w.B + b) * w.T + t0 + t) * w.G + g) * w.N + n;
                w.part_b[to] = sb;
                w.part_c[to] = sc;
            }
        }
    };

    if (n_chunk > 0) {
        fetch(t_start);
        stage(t_start, n_chunk - 1 & 1);
        if (n_chunk > 1) fetch(t_start - kK);
    }
    // dskip and ddt_bias, of sums over 64 of this thread's tokens: one long chain would lose digits.  (Kept in shared memory,
    // and added outside the loop below: with a condition inside it a training step takes 10 % longer.)
    float4 &sums = sm.sums[tid];
    sums = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add_up = [&]() {
        sums.x += dskip[0], sums.y += dskip[1], sums.z += dbias[0], sums.w += dbias[1];
        dskip[0] = dskip[1] = dbias[0] = dbias[1] = 0.f;
    };
    meet();
    for (int k = n_chunk - 1, t0 = t_start; k >= 0; add_up()) {
        do {
            if (k + 1 < n_chunk) finish(t0 + kK, k + 1 & 1, last);
            if (k > 0) {
                stage(t0 - kK, k - 1 & 1);
                if (k > 1) fetch(t0 - 2 * kK);
            }
            meet();
            t0 -= kK;
        } while ((k-- & 63) != 0);
    }
    if (n_chunk > 0) finish(t_first, 0, now);
    add_up();
    {  // nothing stands behind a sequence
        const long long out = static_cast<long long>(b) * w.T * w.D + ld;
        for (int t = max(t_len, t_first) + lt; t < t_end && sub == 0; t += LT) {
            const long long to = out + static_cast<long long>(t) * w.D;
            store_pair<VEC>(static_cast<T *>(w.dx) + to, 0ull, have);
            store_pair<VEC>(static_cast<T *>(w.ddt) + to, 0ull, have);
            if (gated) store_pair<VEC>(static_cast<T *>(w.dgate) + to, 0ull, have);
        }
    }
    asm volatile("bar.sync 2, %0;" ::"n"(kThr) : "memory");
    if (tid < CH / 2) {
        float4 s = sums;
#pragma unroll
        for (int i = 1; i < LT * SUB; ++i) {
            const float4 u = sm.sums[tid + i * (CH / 2)];
            s.x += u.x, s.y += u.y, s.z += u.z, s.w += u.w;
        }
        float *to = part + static_cast<long long>(w.D) * w.N + ld;
        if (have > 0) to[0] = s.x, to[w.D] = s.z;
        if (have > 1) to[1] = s.y, to[w.D + 1] = s.w;
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
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    // taking registers that the launch has not got would wait for ever
    static const int regs = [kernel] {
        cudaFuncAttributes f{};
        return cudaFuncGetAttributes(&f, kernel) == cudaSuccess ? f.numRegs : 0;
    }();
    if (regs != kRegs) return cudaErrorInvalidDeviceFunction;
    kernel<<<static_cast<unsigned>(ss_backward_tiles(a)) * a.G * a.n_seg * a.B, 2 * kThr, bytes, s>>>(a);
    return cudaGetLastError();
}
// eight lanes even where four or two would hold the states: those have more tokens to a preparing thread than registers for
// them (8 states: 69 us per million tokens and channels against 42)
int lanes(int N) { return N <= 16 ? 8 : N <= 32 ? 16 : 32; }
template <typename T, bool VEC>
cudaError_t launch_of(const SsArgs &a, cudaStream_t s) {
    switch (lanes(a.N)) {
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
