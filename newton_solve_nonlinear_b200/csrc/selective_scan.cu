// selective_scan.cu -- the selective scan forward, its time segments, and its single-token step (sm_100a).
// The recurrence is in selective_scan.cuh.
#include <algorithm>

#include "selective_scan.cuh"

namespace pararnn {
using namespace ss;
namespace {

constexpr int kThr = 128;  // threads that hold states; as many again prepare and finish tokens
constexpr int tokens_of(int L) { return L >= 4 ? 16 : 8; }  // between two barriers

enum Pass { kOutputs, kSums, kStates, kReverseSums };

template <int S, int L, bool OUT>
struct SweepSmem {  // two of each, for chunks in turn
    static constexpr int TC = tokens_of(L), CH = 2 * kThr / L, NP = S * L;
    float4 du[2][TC][CH / 2];  // s and s x of two channels (reversed: s and v)
    float b[2][TC][NP], c[OUT ? 2 : 1][OUT ? TC : 1][NP];
    float2 y[OUT ? 2 : 1][OUT ? TC : 1][kThr];
};

// all threads of the CTA, which come from different places of the code
__device__ __forceinline__ void meet() { asm volatile("bar.sync 1, %0;" ::"n"(2 * kThr) : "memory"); }

// One CTA: 2 kThr / L channels of one group, one segment of one sequence, in chunks of TC tokens.
//   Four warps hold the states: a thread has S states of each of two channels, so that what it reads of b and c from shared
// memory serves both (every lane's bytes count there, the same address or not: with one channel to a thread these reads took
// as long as the arithmetic); L lanes share the two channels.
//   Four more prepare the next chunk (s and s x of each token and channel; VEC: pairs of channels, and quads of b and c, lie
// on their own alignment) and finish the last one (the sum over the lanes, skip, gate), in the gaps that the chains of
// dependent operations leave the others.
//   Bound by instructions, 13 to a state, issued in 61 % of the cycles: 8 x 4096 x 2048 x 16 in bf16 680 us, where the
// exponentials alone take 239 and the bytes 82.  (Preparing and finishing in the states' own warps: 762.)
//   kOutputs      from the start state: y, the kept states, and the last segment's last state
//   kStates       from the start state: the kept states alone
//   kSums         from zero: the segment's last state and sum of s
//   kReverseSums  from zero, backward in time: P before the segment
template <typename T, int S, int L, Pass PASS, bool VEC>
__global__ void __launch_bounds__(2 * kThr, 2) ss_sweep_kernel(const SsArgs w) {
    constexpr bool OUT = PASS == kOutputs, REV = PASS == kReverseSums, SUMS = PASS == kSums || REV;
    using SM = SweepSmem<S, L, OUT>;
    constexpr int TC = SM::TC, CH = SM::CH, NP = SM::NP, Q = S / 2;  // Q pairs of states
    extern __shared__ __align__(16) char smem[];
    SM &sm = *reinterpret_cast<SM *>(smem);

    const int per = w.D / w.G, tiles = (per + CH - 1) / CH, blocks = tiles * w.G;
    const int tile = blockIdx.x % blocks % tiles, g = blockIdx.x % blocks / tiles;
    const int seg = blockIdx.x / blocks % w.n_seg, b = blockIdx.x / blocks / w.n_seg;
    const int len = row_count(w.lengths, b, w.T);
    const int t_first = seg * w.seg, t_end = min(w.T, t_first + w.seg), t_len = min(t_end, len);
    const int n_chunk = (max(t_len - t_first, 0) + TC - 1) / TC;
    const int t_start = t_first + (REV ? max(n_chunk - 1, 0) * TC : 0);  // the chunks go on from here, TC tokens at a time
    constexpr int STEP = REV ? -TC : TC;

    if (threadIdx.x < kThr) {
        const int tid = threadIdx.x, pair = tid / L, n0 = tid % L * S, d = g * per + tile * CH + 2 * pair;
        const int owns = min(2, max(0, per - tile * CH - 2 * pair));
        const bool vec = w.N % S == 0;
        const long long at_d = (static_cast<long long>(b) * w.D + d) * w.N, all = static_cast<long long>(w.B) * w.D * w.N;
        u64 h[2][Q] = {};
        float a[2][S] = {};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (q >= owns) continue;
#pragma unroll
            for (int i = 0; i < S; ++i)
                if (n0 + i < w.N) a[q][i] = rate_of(w.a[(static_cast<long long>(d) + q) * w.N + n0 + i]);
            if (!SUMS) {
                const float *from = w.n_seg > 1 ? w.seg_state + seg * all : w.h0;
                if (from != nullptr) load_states(h[q], from + at_d + q * w.N, n0, w.N, vec);
            }
        }
        const long long row = static_cast<long long>(w.D) * w.N;
        float *kept = SUMS || w.kept == nullptr
                          ? nullptr
                          : w.kept + (static_cast<long long>(b) * ((w.T + kSsKeep - 1) / kSsKeep) + t_start / kSsKeep) * row +
                                static_cast<long long>(d) * w.N;
        meet();
        for (int k = 0, t0 = t_start; k < n_chunk; ++k, t0 += STEP) {
            const auto &du_at = sm.du[k & 1];
            const auto &b_at = sm.b[k & 1];
            const auto &c_at = sm.c[OUT ? k & 1 : 0];
            auto &y_at = sm.y[OUT ? k & 1 : 0];
#pragma unroll 1
            for (int j0 = 0; j0 < TC; j0 += kSsKeep) {
                if (!SUMS && kept != nullptr) {
                    if (t0 + j0 < t_len) {
                        if (owns > 0) store_states(h[0], kept, n0, w.N, vec);
                        if (owns > 1) store_states(h[1], kept + w.N, n0, w.N, vec);
                    }
                    kept += row;
                }
#pragma unroll
                for (int j = 0; j < kSsKeep; ++j) {
                    const int t = REV ? TC - 1 - j0 - j : j0 + j;
                    const float4 du = du_at[t][pair];
                    u64 bb[Q], cc[Q];
                    float y[2];
                    load_pairs(bb, &b_at[t][n0]);
                    if (OUT) load_pairs(cc, &c_at[t][n0]);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float st = q == 0 ? du.x : du.y, u = q == 0 ? du.z : du.w;
                        u64 part = 0;
#pragma unroll
                        for (int i = 0; i < Q; ++i) {
                            const u64 xx = pk(st * a[q][2 * i], st * a[q][2 * i + 1]), f = decay_factor(xx);
                            // one factor for both of a pair: two instructions, as moving it beside itself would take
                            float b0, b1, h0, h1;
                            upk(bb[i], b0, b1), upk(h[q][i], h0, h1);
                            if constexpr (REV) {
                                const u64 moved = pk(fmaf(u, b0, h0), fmaf(u, b1, h1));
                                upk(mul2(f, moved), h0, h1);
                                h[q][i] = with_rest(xx, h0, h1, moved);
                            } else {
                                h[q][i] = fma2(f, h[q][i], with_rest(xx, u * b0, u * b1, h[q][i]));
                            }
                            if (OUT) part = i == 0 ? mul2(cc[i], h[q][i]) : fma2(cc[i], h[q][i], part);
                        }
                        if (OUT) y[q] = pair_sum(part);
                    }
                    if (OUT) y_at[t][tid] = make_float2(y[0], y[1]);
                }
            }
            meet();
        }
        float *last = SUMS ? (REV ? w.rev_state : w.seg_state) + seg * all : w.h;
        if (SUMS || (OUT && seg == w.n_seg - 1)) {
            if (owns > 0) store_states(h[0], last + at_d, n0, w.N, vec);
            if (owns > 1) store_states(h[1], last + at_d + w.N, n0, w.N, vec);
        }
        return;
    }

    // tokens lt + i LT of a chunk, channels lc and lc + 1
    constexpr int LT = kThr / (CH / 2), PER = (TC + LT - 1) / LT;
    const int tid = threadIdx.x - kThr;
    const int lc = tid % (CH / 2) * 2, lt = tid / (CH / 2), ld = g * per + tile * CH + lc;
    const int have = min(2, max(0, per - tile * CH - lc));
    float bias[2] = {}, skip[2] = {};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        if (q < have && w.dt_bias != nullptr) bias[q] = w.dt_bias[ld + q];
        if (OUT && q < have && w.skip != nullptr) skip[q] = w.skip[ld + q];
    }
    const bool gated = w.gate.p != nullptr;
    const SsRows &rx = REV ? w.dy : w.x, &rb = REV ? w.c : w.b;
    // where this thread's next elements are
    const T *px = static_cast<const T *>(rx.p) + b * rx.sb + ld + (t_start + lt) * rx.st;
    const T *pdt = static_cast<const T *>(w.dt.p) + b * w.dt.sb + ld + (t_start + lt) * w.dt.st;
    const T *pg = static_cast<const T *>(w.gate.p) + b * w.gate.sb + ld + (t_start + lt) * w.gate.st;
    constexpr int BW = VEC ? 4 : 1, BROW = NP / BW, NB = (TC * BROW + kThr - 1) / kThr;  // of b and c, BW at a time
    const int bt = tid / BROW, bn = tid % BROW * BW;
    const T *pb = static_cast<const T *>(rb.p) + b * rb.sb + g * rb.sg + (t_start + bt) * rb.st + bn;
    const T *pc = static_cast<const T *>(w.c.p) + b * w.c.sb + g * w.c.sg + (t_start + bt) * w.c.st + bn;
    T *py = static_cast<T *>(w.y) + (static_cast<long long>(b) * w.T + t_start + lt) * w.D + ld;

    Raw<T> nx[PER], ndt[PER], ng[PER], cx[PER], cg[PER], ox[PER], og[PER];  // of the next chunk, the present and the last one
    RawN<T, BW> nb[NB], nc[NB];
    u64 sum = 0;
    auto fetch = [&](int t0) {
        const int left = t_len - t0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = lt + i * LT, n = t < TC && t < left ? have : 0;
            nx[i] = load_raw<VEC>(px + i * LT * rx.st, n);
            ndt[i] = load_raw<VEC>(pdt + i * LT * w.dt.st, n);
            if (OUT || REV) ng[i] = load_raw<VEC>(pg + i * LT * w.gate.st, gated ? n : 0);
        }
        px += STEP * rx.st, pdt += STEP * w.dt.st, pg += STEP * w.gate.st;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int t = bt + i * (kThr / BROW);
            const bool on = t < TC && t < left && bn < w.N;
            nb[i] = load_n<BW>(pb + i * (kThr / BROW) * rb.st, on);
            if (OUT) nc[i] = load_n<BW>(pc + i * (kThr / BROW) * w.c.st, on);
        }
        pb += STEP * rb.st, pc += STEP * w.c.st;
    };
    // (each step for all of the thread's tokens before the next step: chains of dependent operations side by side)
    auto stage = [&](int t0, int to) {
        float st[PER][2], u[PER][2];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            upk(value(ndt[i]), st[i][0], st[i][1]);
            st[i][0] += bias[0], st[i][1] += bias[1];
        }
        if (w.softplus) {
#pragma unroll
            for (int i = 0; i < PER; ++i) st[i][0] = softplus(st[i][0]), st[i][1] = softplus(st[i][1]);
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool on = t0 + lt + i * LT < t_len;
            st[i][0] = on ? st[i][0] : 0.f, st[i][1] = on ? st[i][1] : 0.f;
            upk(value(nx[i]), u[i][0], u[i][1]);
            if (!REV) u[i][0] *= st[i][0], u[i][1] *= st[i][1];
        }
        if (REV && gated) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                float z[2];
                upk(value(ng[i]), z[0], z[1]);
                u[i][0] = gate_with(u[i][0], z[0]), u[i][1] = gate_with(u[i][1], z[1]);
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = lt + i * LT;
            if (t < TC) {
                sm.du[to][t][lc / 2] = make_float4(st[i][0], st[i][1], u[i][0], u[i][1]);
                if (SUMS) sum = add2(sum, pk(st[i][0], st[i][1]));
            }
            if (OUT) ox[i] = cx[i], og[i] = cg[i], cx[i] = nx[i], cg[i] = ng[i];
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int t = bt + i * (kThr / BROW);
            if (t < TC) {
                store_n(&sm.b[to][t][bn], nb[i]);
                if (OUT) store_n(&sm.c[to][t][bn], nc[i]);
            }
        }
    };
    auto finish = [&](int t0, int from, const Raw<T> (&x)[PER], const Raw<T> (&z)[PER]) {
        float y[PER][2];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            float part[2 * L], v[2];
            upk(value(x[i]), v[0], v[1]);
            load_floats<2 * L>(part, &sm.y[from][min(lt + i * LT, TC - 1)][lc / 2 * L].x);
#pragma unroll
            for (int q = 1; q < L; ++q) part[0] += part[2 * q], part[1] += part[2 * q + 1];
            y[i][0] = fmaf(skip[0], v[0], part[0]), y[i][1] = fmaf(skip[1], v[1], part[1]);
        }
        if (gated) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                float g2[2];
                upk(value(z[i]), g2[0], g2[1]);
                y[i][0] = gate_with(y[i][0], g2[0]), y[i][1] = gate_with(y[i][1], g2[1]);
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = lt + i * LT;
            store_pair<VEC>(py + static_cast<long long>(i * LT) * w.D, pk(y[i][0], y[i][1]), t < TC && t0 + t < t_len ? have : 0);
        }
        py += static_cast<long long>(TC) * w.D;
    };

    if (n_chunk > 0) {
        fetch(t_start);
        stage(t_start, 0);
        if (n_chunk > 1) fetch(t_start + STEP);
    }
    meet();
    for (int k = 0, t0 = t_start; k < n_chunk; ++k, t0 += STEP) {
        if (OUT && k > 0) finish(t0 - TC, k - 1 & 1, ox, og);
        if (k + 1 < n_chunk) {
            stage(t0 + STEP, k + 1 & 1);
            if (k + 2 < n_chunk) fetch(t0 + 2 * STEP);
        }
        meet();
    }
    if (OUT) {
        if (n_chunk > 0) finish(t_start + (n_chunk - 1) * TC, n_chunk - 1 & 1, cx, cg);
        // nothing stands behind a sequence
        py = static_cast<T *>(w.y) + static_cast<long long>(b) * w.T * w.D + ld;
        for (int t = max(t_len, t_first) + lt; t < t_end; t += LT) store_pair<VEC>(py + static_cast<long long>(t) * w.D, 0ull, have);
    }
    if (SUMS) {
        u64 *s_sum = reinterpret_cast<u64 *>(smem);  // the states' threads are done with it
        s_sum[tid] = sum;
        asm volatile("bar.sync 2, %0;" ::"n"(kThr) : "memory");
        if (tid < CH / 2) {
            u64 s = 0;
#pragma unroll
            for (int i = 0; i < LT; ++i) s = add2(s, s_sum[tid + i * (CH / 2)]);
            float s0, s1;
            upk(s, s0, s1);
            float *to = w.seg_dt + (static_cast<long long>(seg) * w.B + b) * w.D + ld;
            if (have > 0) to[0] = s0;
            if (have > 1) to[1] = s1;
        }
    }
}

// Each segment's own last state becomes the state that it starts from; REV: from the last segment to the first.
template <bool REV>
__global__ void ss_join_kernel(const SsArgs w) {
    const long long all = static_cast<long long>(w.B) * w.D * w.N;
    const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= all) return;
    const long long bd = i / w.N;
    const float a = above_inf(w.a[bd % w.D * w.N + i % w.N]);
    const float *first = REV ? w.dh : w.h0;
    float *at = (REV ? w.rev_state : w.seg_state) + i;
    float h = first == nullptr ? 0.f : first[i];
    for (int k = 0; k < w.n_seg; ++k) {
        const int seg = REV ? w.n_seg - 1 - k : k;
        // (both loads before the store and outside of the condition: a step of this chain is their latency)
        const float own = at[seg * all], decay = expf(a * w.seg_dt[seg * (all / w.N) + bd]);
        at[seg * all] = h;
        // a state that is zero stays so, whatever a segment's growth: infinity times zero would be NaN
        const float kept = h == 0.f ? 0.f : decay;
        h = fmaf(kept, h, own);
    }
}

// Lanes of a channel: as many as its states take, four to each, or two where there are too few warps otherwise.
struct Lanes {
    int s, l;
};
Lanes lanes_of(int N, int s) {
    int l = 2;
    while (l * s < N) l *= 2;
    return {s, l};
}
long long ctas(const SsArgs &a, Lanes f) {
    const int per = a.D / a.G, ch = 2 * kThr / f.l;
    return static_cast<long long>((per + ch - 1) / ch) * a.G * a.B;
}
Lanes lanes_for(const SsArgs &a) {
    const Lanes four = lanes_of(a.N, 4);
    return ctas(a, four) * a.n_seg < 100 && a.N > 2 ? lanes_of(a.N, 2) : four;
}
template <typename T, int S, int L, Pass PASS, bool VEC>
cudaError_t launch_pass(const SsArgs &a, cudaStream_t s) {
    const auto kernel = ss_sweep_kernel<T, S, L, PASS, VEC>;
    constexpr int bytes = sizeof(SweepSmem<S, L, PASS == kOutputs>);
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    kernel<<<static_cast<unsigned>(ctas(a, {S, L}) * a.n_seg), 2 * kThr, bytes, s>>>(a);
    return cudaGetLastError();
}
template <typename T, int S, int L, bool VEC>
cudaError_t launch_sweep(const SsArgs &a, Pass pass, cudaStream_t s) {
    if (pass == kOutputs) return launch_pass<T, S, L, kOutputs, VEC>(a, s);
    if (pass == kSums) return launch_pass<T, S, L, kSums, VEC>(a, s);
    if (pass == kStates) return launch_pass<T, S, L, kStates, VEC>(a, s);
    return launch_pass<T, S, L, kReverseSums, VEC>(a, s);
}
template <typename T, bool VEC>
cudaError_t sweep_of(const SsArgs &a, Pass pass, cudaStream_t s) {
    const Lanes f = lanes_for(a);
#define PARARNN_SS(S_, L_) \
    if (f.s == S_ && f.l == L_) return launch_sweep<T, S_, L_, VEC>(a, pass, s)
    PARARNN_SS(4, 2);
    PARARNN_SS(4, 4);
    PARARNN_SS(4, 8);
    PARARNN_SS(4, 16);
    PARARNN_SS(2, 2);
    PARARNN_SS(2, 4);
    PARARNN_SS(2, 8);
    PARARNN_SS(2, 16);
    PARARNN_SS(2, 32);
#undef PARARNN_SS
    return cudaErrorInvalidValue;
}
cudaError_t sweep(const SsArgs &a, Pass pass, cudaStream_t s) {
    const bool vec = ss_pairs_ok(a);
    if (a.dtype == PARARNN_F32) return vec ? sweep_of<float, true>(a, pass, s) : sweep_of<float, false>(a, pass, s);
    return vec ? sweep_of<__nv_bfloat16, true>(a, pass, s) : sweep_of<__nv_bfloat16, false>(a, pass, s);
}
cudaError_t join(const SsArgs &a, bool reverse, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>((static_cast<long long>(a.B) * a.D * a.N + 255) / 256);
    if (reverse) ss_join_kernel<true><<<grid, 256, 0, s>>>(a);
    else ss_join_kernel<false><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError();
}
cudaError_t start_states(const SsArgs &a, cudaStream_t s) {
    if (a.n_seg == 1) return cudaSuccess;
    const cudaError_t e = sweep(a, kSums, s);
    return e != cudaSuccess ? e : join(a, false, s);
}

}  // namespace

bool ss_pairs_ok(const SsArgs &a) {
    const size_t e = a.dtype == PARARNN_F32 ? 8 : 4;
    bool ok = a.D / a.G % 2 == 0 && a.N % 4 == 0;
    for (const SsRows *r : {&a.b, &a.c})
        ok = ok && reinterpret_cast<uintptr_t>(r->p) % (2 * e) == 0 && r->sb % 4 == 0 && r->st % 4 == 0 && r->sg % 4 == 0;
    for (const SsRows *r : {&a.x, &a.dt, &a.gate, &a.dy})
        ok = ok && reinterpret_cast<uintptr_t>(r->p) % e == 0 && r->sb % 2 == 0 && r->st % 2 == 0;
    return ok;
}

// Segments: none where two states to a thread fill two thirds of the SMs, since what they cost is a second pass; otherwise as
// many as it takes to give every SM two CTAs at once, of at least 64 tokens each.
SsPlan ss_plan(const SsArgs &a) {
    const long long most = ctas(a, lanes_of(a.N, a.N > 2 ? 2 : 4)), have = ctas(a, lanes_of(a.N, 4));
    const long long want = most >= 100 ? 1 : std::min<long long>(148 * 2 / have, (a.T + 63) / 64);
    if (want < 2) return {1, a.T};
    const int seg = static_cast<int>(((a.T + want - 1) / want + 15) / 16 * 16);
    return {(a.T + seg - 1) / seg, seg};
}

cudaError_t launch_ss_forward(const SsArgs &a, cudaStream_t s) {
    const cudaError_t e = start_states(a, s);
    return e != cudaSuccess ? e : sweep(a, kOutputs, s);
}
cudaError_t launch_ss_kept(const SsArgs &a, cudaStream_t s) {
    const cudaError_t e = start_states(a, s);
    return e != cudaSuccess ? e : sweep(a, kStates, s);
}
cudaError_t launch_ss_reverse_states(const SsArgs &a, cudaStream_t s) {
    if (a.n_seg == 1) return cudaSuccess;
    const cudaError_t e = sweep(a, kReverseSums, s);
    return e != cudaSuccess ? e : join(a, true, s);
}

// ---- one token per sequence ---------------------------------------------------------------------------------

namespace {

// CTAs along the channels of each row; L lanes of four states hold a channel, each thread of R channels that stand CH apart,
// of which it prepares and finishes one (the lanes take turns).  Everything that a row needs is asked for at once, behind its
// slot alone.  Rows that name the same slot are taken in row order by the first one's CTA, as tokens that follow each other.
// 256 rows of 4096 channels of 16: 45 us, 0.48 of HBM's rate; issue slots 73 % busy with 63 instructions to a state, most of them
// the row's and the channel's own (one channel to a thread, prepared by all of its lanes, with its loads in four steps: 83).
template <typename T, int L, int R, bool VEC>
__global__ void __launch_bounds__(256) ss_step_kernel(const SsStep w) {
    constexpr int CH = 256 / L, BW = VEC ? 4 : 1;
    __shared__ int next;
    const int tid = threadIdx.x, tiles = (w.D + CH * R - 1) / (CH * R);
    int b = blockIdx.x / tiles;
    const int d0 = blockIdx.x % tiles * CH * R + tid / L, n0 = tid % L * 4, per = w.D / w.G;
    T *py = static_cast<T *>(w.y);
    const int slot = w.slots == nullptr ? b : w.slots[b];
    if (slot < 0 || slot >= w.n_slots) {  // no state behind this row
        for (int r = 0; r < R; ++r)
            if (d0 + r * CH < w.D && n0 == 0) py[static_cast<long long>(b) * w.D + d0 + r * CH] = from_f<T>(0.f);
        return;
    }
    const bool vec = w.N % 4 == 0, vec_a = vec && (reinterpret_cast<uintptr_t>(w.a) & 15) == 0;
    const long long at = (static_cast<long long>(slot) * w.D + d0) * w.N;
    static_assert(R <= L, "a lane for each channel");
    const int mine = R == 1 ? 0 : tid & 1, dm = d0 + mine * CH;
    u64 h[R][2] = {}, a[R][2] = {};
    float bias = 0.f, skip = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int d = d0 + r * CH;
        if (d >= w.D) continue;
        load_states(h[r], w.state + at + static_cast<long long>(r) * CH * w.N, n0, w.N, vec);
        load_states(a[r], w.a + static_cast<long long>(d) * w.N, n0, w.N, vec_a);
    }
    if (dm < w.D && w.dt_bias != nullptr) bias = w.dt_bias[dm];
    if (dm < w.D && w.skip != nullptr) skip = w.skip[dm];
    T x, s, z;
    RawN<T, BW> rb[R][4 / BW], rc[R][4 / BW];
    auto fetch = [&]() {
        x = s = z = from_f<T>(0.f);
        if (dm < w.D) {
            x = static_cast<const T *>(w.x.p)[b * w.x.sb + dm], s = static_cast<const T *>(w.dt.p)[b * w.dt.sb + dm];
            if (w.gate.p != nullptr) z = static_cast<const T *>(w.gate.p)[b * w.gate.sb + dm];
        }
        const T *pb = static_cast<const T *>(w.b.p) + b * w.b.sb + n0, *pc = static_cast<const T *>(w.c.p) + b * w.c.sb + n0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int d = d0 + r * CH;
            const bool on = d < w.D;
            if (r > 0 && w.G == 1) {  // one group: the same b and c
#pragma unroll
                for (int i = 0; i < 4 / BW; ++i) rb[r][i] = rb[0][i], rc[r][i] = rc[0][i];
                continue;
            }
            const int g = on && w.G > 1 ? d / per : 0;
#pragma unroll
            for (int i = 0; i < 4 / BW; ++i) {
                rb[r][i] = load_n<BW>(pb + g * w.b.sg + i * BW, on && n0 + i * BW < w.N);
                rc[r][i] = load_n<BW>(pc + g * w.c.sg + i * BW, on && n0 + i * BW < w.N);
            }
        }
    };
    auto token = [&]() {
        const float xf = to_f(x);
        float st = to_f(s) + bias, out[R];
        if (w.softplus) st = softplus(st);
        const float u = st * xf;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int from = R == 1 ? tid & 31 : (tid & 30) | r;
            const u64 st2 = splat(__shfl_sync(0xffffffffu, st, from)), u2 = splat(__shfl_sync(0xffffffffu, u, from));
            float bf[4], cf[4];
#pragma unroll
            for (int i = 0; i < 4 / BW; ++i) unpack_n(bf + i * BW, rb[r][i]), unpack_n(cf + i * BW, rc[r][i]);
            u64 y = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const u64 xx = mul2(st2, a[r][i]);
                float b0, b1;
                upk(mul2(u2, pk(bf[2 * i], bf[2 * i + 1])), b0, b1);
                h[r][i] = fma2(decay_factor(xx), h[r][i], with_rest(xx, b0, b1, h[r][i]));
                y = i == 0 ? mul2(pk(cf[0], cf[1]), h[r][0]) : fma2(pk(cf[2], cf[3]), h[r][1], y);
            }
            out[r] = pair_sum(y);
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) out[r] += __shfl_xor_sync(0xffffffffu, out[r], o);
        }
        float v = fmaf(skip, xf, mine == 0 ? out[0] : out[R - 1]);
        if (w.gate.p != nullptr) v = gate_with(v, to_f(z));
        if (dm < w.D && tid % L < R) py[static_cast<long long>(b) * w.D + dm] = from_f<T>(v);
    };
    fetch();
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float a0, a1;
            upk(a[r][i], a0, a1);
            a[r][i] = pk(rate_of(a0), rate_of(a1));
        }
    bool more = false;
    if (w.slots != nullptr) {
        int earlier = 0, later = 0;
        for (int i = tid; i < w.B; i += 256) {
            const int same = w.slots[i] == slot;
            earlier |= same & i < b, later |= same & i > b;
        }
        if (__syncthreads_or(earlier)) return;
        more = __syncthreads_or(later);
    }
    token();
    while (more) {
        if (tid == 0) next = w.B;
        __syncthreads();
        for (int i = b + 1 + tid; i < w.B; i += 256)
            if (w.slots[i] == slot) {
                atomicMin(&next, i);
                break;
            }
        __syncthreads();
        b = next;
        if (b >= w.B) break;
        __syncthreads();
        fetch();
        token();
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (d0 + r * CH < w.D) store_states(h[r], w.out_state + at + static_cast<long long>(r) * CH * w.N, n0, w.N, vec);
}

template <typename T, int L>
void launch_step(const SsStep &w, cudaStream_t s) {
    constexpr int CH = 256 / L;
    const long long one = static_cast<long long>((w.D + CH - 1) / CH) * w.B;
    const size_t e = 4 * sizeof(T);
    bool quads = w.N % 4 == 0;
    for (const SsRows *r : {&w.b, &w.c})
        quads = quads && reinterpret_cast<uintptr_t>(r->p) % e == 0 && r->sb % 4 == 0 && r->sg % 4 == 0;
    const unsigned two = static_cast<unsigned>((w.D + 2 * CH - 1) / (2 * CH)) * w.B;
    if (!quads) ss_step_kernel<T, L, 1, false><<<static_cast<unsigned>(one), 256, 0, s>>>(w);
    // one channel to a thread while that is little more than a wave (five of these CTAs fit an SM): 256 CTAs 2.6 us against 2.7
    // with two, 704 3.7 against 3.3, 896 4.9 against 3.8
    else if (L == 1 || one <= 148 * 6) ss_step_kernel<T, L, 1, true><<<static_cast<unsigned>(one), 256, 0, s>>>(w);
    else ss_step_kernel<T, L, L == 1 ? 1 : 2, true><<<two, 256, 0, s>>>(w);
}
template <typename T>
void step_of(const SsStep &w, cudaStream_t s) {
    switch (w.N <= 4 ? 1 : lanes_of(w.N, 4).l) {
        case 1: return launch_step<T, 1>(w, s);
        case 2: return launch_step<T, 2>(w, s);
        case 4: return launch_step<T, 4>(w, s);
        case 8: return launch_step<T, 8>(w, s);
        default: return launch_step<T, 16>(w, s);
    }
}

}  // namespace

cudaError_t launch_ss_step(const SsStep &w, cudaStream_t s) {
    if (w.dtype == PARARNN_F32) step_of<float>(w, s);
    else step_of<__nv_bfloat16>(w, s);
    return cudaGetLastError();
}

}  // namespace pararnn
