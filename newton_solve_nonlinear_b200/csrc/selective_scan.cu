// selective_scan.cu -- the selective scan forward, its time segments, and its single-token step (sm_100a).
// The recurrence is in selective_scan.cuh.
#include <algorithm>

#include "selective_scan.cuh"

namespace pararnn {
using namespace ss;
namespace {

constexpr int kThr = 128;
constexpr int kS = 4;     // states of a thread
constexpr int kTC = 16;   // tokens between two barriers

enum Pass { kOutputs, kSums, kStates, kReverseSums };

// One CTA: kThr / L channels of one group, one segment of one sequence; L lanes of four states each hold a channel.
// Tokens come in chunks of kTC: between two barriers every thread prepares (token, channel) pairs for all (s and s x, by
// element loads that ask nothing of strides or alignment, along the channels so that they coalesce), then runs its states
// through the chunk.
//   kOutputs      from the start state: y, the kept states, and the last segment's last state
//   kStates       from the start state: the kept states alone
//   kSums         from zero: the segment's last state and sum of s
//   kReverseSums  from zero, backward in time: P before the segment
template <typename T, int L, Pass PASS>
__global__ void __launch_bounds__(kThr) ss_sweep_kernel(const SsArgs w) {
    constexpr int CH = kThr / L, NP = kS * L, PER = kTC / L;  // PER: tokens that a thread prepares per chunk
    constexpr bool OUT = PASS == kOutputs, REV = PASS == kReverseSums, SUMS = PASS == kSums || REV;
    __shared__ float4 s_du[kTC][CH];                       // s, s, s x, s x (REV: v, v)
    __shared__ __align__(16) float s_b[kTC][NP], s_c[OUT ? kTC : 1][NP];
    __shared__ __align__(16) float s_y[OUT ? kTC : 1][kThr];
    __shared__ float s_sum[SUMS ? kThr : 1];

    const int tid = threadIdx.x, per = w.D / w.G;
    const int tiles = (per + CH - 1) / CH, blocks = tiles * w.G;
    const int tile = blockIdx.x % blocks % tiles, g = blockIdx.x % blocks / tiles;
    const int seg = blockIdx.x / blocks % w.n_seg, b = blockIdx.x / blocks / w.n_seg;
    const int len = row_count(w.lengths, b, w.T);
    const int t_first = seg * w.seg, t_end = min(w.T, t_first + w.seg), t_len = min(t_end, len);

    // as owner of states
    const int ch = tid / L, n0 = tid % L * kS, d = g * per + tile * CH + ch;
    const bool owner = tile * CH + ch < per;
    const bool vec = w.N % 4 == 0;
    const long long state_at = (static_cast<long long>(b) * w.D + d) * w.N;
    const long long all = static_cast<long long>(w.B) * w.D * w.N;
    u64 h[2] = {0, 0}, a[2] = {0, 0};
    if (owner) {
        load_states(a, w.a + static_cast<long long>(d) * w.N, n0, w.N, false);
#pragma unroll
        for (int i = 0; i < 2; ++i) a[i] = mul2(a[i], splat(kLog2eF));
        if (!SUMS) {
            const float *from = w.n_seg > 1 ? w.seg_state + seg * all : w.h0;
            if (from != nullptr) load_states(h, from + state_at, n0, w.N, false);
        }
    }
    // as the one who prepares tokens t0 + lt + i L of channel lch
    const int lch = tid % CH, lt = tid / CH, ld = g * per + tile * CH + lch;
    const bool loads = tile * CH + lch < per;
    const float bias = loads && w.dt_bias != nullptr ? w.dt_bias[ld] : 0.f;
    const float skip = OUT && loads && w.skip != nullptr ? w.skip[ld] : 0.f;
    const bool gated = w.gate.p != nullptr;
    const T *px = static_cast<const T *>(REV ? w.dy.p : w.x.p) + b * (REV ? w.dy.sb : w.x.sb) + ld;
    const long long stx = REV ? w.dy.st : w.x.st;
    const T *pdt = static_cast<const T *>(w.dt.p) + b * w.dt.sb + ld;
    const T *pg = static_cast<const T *>(w.gate.p) + b * w.gate.sb + ld;
    const SsRows &rb = REV ? w.c : w.b;
    const T *pb = static_cast<const T *>(rb.p) + b * rb.sb + g * rb.sg;
    const T *pc = static_cast<const T *>(w.c.p) + b * w.c.sb + g * w.c.sg;
    constexpr int NB = kTC * NP / kThr;  // elements of b that a thread brings per chunk (kS * kTC * L / kThr)
    constexpr int NBE = NB > 0 ? NB : 1;

    float nx[PER], ndt[PER], ng[PER], cx[PER], cg[PER], nb[NBE], nc[NBE], sum = 0.f;
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = t0 + lt + i * L;
            const bool on = loads && t < t_len;
            nx[i] = on ? to_f(px[t * stx]) : 0.f;
            ndt[i] = on ? to_f(pdt[t * w.dt.st]) : 0.f;
            if (OUT || REV) ng[i] = on && gated ? to_f(pg[t * w.gate.st]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < NBE; ++i) {
            const int e = tid + i * kThr, t = t0 + e / NP, n = e % NP;
            const bool on = e < kTC * NP && n < w.N && t < t_len;
            nb[i] = on ? to_f(pb[t * rb.st + n]) : 0.f;
            if (OUT) nc[i] = on ? to_f(pc[t * w.c.st + n]) : 0.f;
        }
    };
    auto stage = [&](int t0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = lt + i * L;
            float s = 0.f, u = 0.f;
            if (loads && t0 + t < t_len) {
                s = ndt[i] + bias;
                if (w.softplus) s = softplus(s);
                if (REV) u = gated ? gate_with(nx[i], ng[i]) : nx[i];
                else u = s * nx[i];
            }
            s_du[t][lch] = make_float4(s, s, u, u);
            if (SUMS) sum += s;
            cx[i] = nx[i], cg[i] = ng[i];
        }
#pragma unroll
        for (int i = 0; i < NBE; ++i) {
            const int e = tid + i * kThr;
            if (e < kTC * NP) {
                s_b[e / NP][e % NP] = nb[i];
                if (OUT) s_c[e / NP][e % NP] = nc[i];
            }
        }
    };

    const int n_chunk = (max(t_len - t_first, 0) + kTC - 1) / kTC;
    auto chunk_at = [&](int k) { return t_first + (REV ? n_chunk - 1 - k : k) * kTC; };
    if (n_chunk > 0) {
        fetch(chunk_at(0));
        stage(chunk_at(0));
    }
    for (int k = 0; k < n_chunk; ++k) {
        const int t0 = chunk_at(k);
        __syncthreads();
        if (k + 1 < n_chunk) fetch(chunk_at(k + 1));
#pragma unroll 4
        for (int j = 0; j < kTC; ++j) {
            const int t = REV ? kTC - 1 - j : j;
            if (!SUMS && (j & (kSsKeep - 1)) == 0 && w.kept != nullptr && owner && t0 + t < t_len)
                store_states(h, w.kept + ((static_cast<long long>(b) * ((w.T + kSsKeep - 1) / kSsKeep) +
                                           (t0 + t) / kSsKeep) * w.D + d) * w.N, n0, w.N, vec);
            const ulonglong2 du = *reinterpret_cast<const ulonglong2 *>(&s_du[t][ch]);
            u64 bb[2], cc[2], y = 0;
            load_pairs(bb, &s_b[t][n0]);
            if (OUT) load_pairs(cc, &s_c[t][n0]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const u64 e = decay_less_one(mul2(du.x, a[i]));
                if (REV) {
                    h[i] = fma2(du.y, bb[i], h[i]);
                    h[i] = fma2(e, h[i], h[i]);
                } else {
                    h[i] = fma2(e, h[i], fma2(du.y, bb[i], h[i]));
                }
                if (OUT) y = fma2(cc[i], h[i], y);
            }
            if (OUT) s_y[t][tid] = pair_sum(y);
        }
        __syncthreads();
        if (OUT) {
            T *py = static_cast<T *>(w.y) + (static_cast<long long>(b) * w.T + t0) * w.D + ld;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int t = lt + i * L;
                float y = 0.f;
#pragma unroll
                for (int j = 0; j < L; ++j) y += s_y[t][lch * L + j];
                y = fmaf(skip, cx[i], y);
                if (gated) y = gate_with(y, cg[i]);
                if (loads && t0 + t < t_len) py[static_cast<long long>(t) * w.D] = from_f<T>(y);
            }
        }
        if (k + 1 < n_chunk) stage(chunk_at(k + 1));
    }
    if (OUT && loads) {  // nothing stands behind a sequence
        T *py = static_cast<T *>(w.y) + static_cast<long long>(b) * w.T * w.D + ld;
        for (int t = max(t_len, t_first) + lt; t < t_end; t += L) py[static_cast<long long>(t) * w.D] = from_f<T>(0.f);
    }
    if (OUT && seg == w.n_seg - 1 && owner) store_states(h, w.h + state_at, n0, w.N, false);
    if (SUMS) {
        if (owner) store_states(h, (REV ? w.rev_state : w.seg_state) + seg * all + state_at, n0, w.N, false);
        s_sum[tid] = sum;
        __syncthreads();
        if (tid < CH && tile * CH + tid < per) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < L; ++i) s += s_sum[tid + i * CH];
            w.seg_dt[(static_cast<long long>(seg) * w.B + b) * w.D + g * per + tile * CH + tid] = s;
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
    const float a = w.a[bd % w.D * w.N + i % w.N];
    const float *first = REV ? w.dh : w.h0;
    float *at = (REV ? w.rev_state : w.seg_state) + i;
    float h = first == nullptr ? 0.f : first[i];
    for (int k = 0; k < w.n_seg; ++k) {
        const int seg = REV ? w.n_seg - 1 - k : k;
        const float own = at[seg * all];
        at[seg * all] = h;
        h = fmaf(expf(a * w.seg_dt[seg * (all / w.N) + bd]), h, own);
    }
}

template <typename T, int L>
void launch_sweep(const SsArgs &a, Pass pass, cudaStream_t s) {
    const int per = a.D / a.G, tiles = (per + kThr / L - 1) / (kThr / L);
    const unsigned grid = static_cast<unsigned>(tiles) * a.G * a.n_seg * a.B;
    if (pass == kOutputs) ss_sweep_kernel<T, L, kOutputs><<<grid, kThr, 0, s>>>(a);
    else if (pass == kSums) ss_sweep_kernel<T, L, kSums><<<grid, kThr, 0, s>>>(a);
    else if (pass == kStates) ss_sweep_kernel<T, L, kStates><<<grid, kThr, 0, s>>>(a);
    else ss_sweep_kernel<T, L, kReverseSums><<<grid, kThr, 0, s>>>(a);
}

int lanes(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

template <typename T>
void sweep_of(const SsArgs &a, Pass pass, cudaStream_t s) {
    switch (lanes(a.N)) {
        case 1: return launch_sweep<T, 1>(a, pass, s);
        case 2: return launch_sweep<T, 2>(a, pass, s);
        case 4: return launch_sweep<T, 4>(a, pass, s);
        case 8: return launch_sweep<T, 8>(a, pass, s);
        default: return launch_sweep<T, 16>(a, pass, s);
    }
}
cudaError_t sweep(const SsArgs &a, Pass pass, cudaStream_t s) {
    if (a.dtype == PARARNN_F32) sweep_of<float>(a, pass, s);
    else sweep_of<__nv_bfloat16>(a, pass, s);
    return cudaGetLastError();
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

// Segments: as many as it takes to give every scheduler of the card about two warps, of at least 64 tokens each.
SsPlan ss_plan(const SsArgs &a, bool) {
    const int per = a.D / a.G, ch = kThr / lanes(a.N);
    const long long ctas = static_cast<long long>((per + ch - 1) / ch) * a.G * a.B;
    long long want = (148 * 2 + ctas - 1) / ctas;
    if (want < 2) return {1, a.T};
    want = std::min<long long>(want, (a.T + 63) / 64);
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

// CTAs along the channels of each row; L lanes of four states hold a channel, each with one vector of the state.  Rows
// that name the same slot are taken in row order by the first one's CTA, as tokens that follow each other.
template <typename T, int L>
__global__ void __launch_bounds__(256) ss_step_kernel(const SsStep w) {
    constexpr int CH = 256 / L;
    __shared__ int next;
    const int tid = threadIdx.x, tiles = (w.D + CH - 1) / CH;
    int b = blockIdx.x / tiles;
    const int d = blockIdx.x % tiles * CH + tid / L, n0 = tid % L * 4, g = d / (w.D / w.G);
    const bool on = d < w.D;
    T *py = static_cast<T *>(w.y);
    const int slot = w.slots == nullptr ? b : w.slots[b];
    if (slot < 0 || slot >= w.n_slots) {  // no state behind this row
        if (on && n0 == 0) py[static_cast<long long>(b) * w.D + d] = from_f<T>(0.f);
        return;
    }
    if (w.slots != nullptr) {
        int earlier = 0;
        for (int i = tid; i < b; i += 256) earlier |= w.slots[i] == slot;
        if (__syncthreads_or(earlier)) return;
    }
    const bool vec = w.N % 4 == 0;
    const long long at = (static_cast<long long>(slot) * w.D + d) * w.N;
    u64 h[2] = {0, 0}, a[2] = {0, 0};
    float bias = 0.f, skip = 0.f;
    if (on) {
        load_states(h, w.state + at, n0, w.N, vec);
        load_states(a, w.a + static_cast<long long>(d) * w.N, n0, w.N, vec && (reinterpret_cast<uintptr_t>(w.a) & 15) == 0);
        if (w.dt_bias != nullptr) bias = w.dt_bias[d];
        if (w.skip != nullptr) skip = w.skip[d];
    }
    while (true) {
        if (w.slots != nullptr) {
            if (tid == 0) next = w.B;
            __syncthreads();
        }
        float x = 0.f, s = 0.f;
        if (on) {
            x = to_f(static_cast<const T *>(w.x.p)[b * w.x.sb + d]);
            s = to_f(static_cast<const T *>(w.dt.p)[b * w.dt.sb + d]) + bias;
            if (w.softplus) s = softplus(s);
        }
        const T *pb = static_cast<const T *>(w.b.p) + b * w.b.sb + g * w.b.sg;
        const T *pc = static_cast<const T *>(w.c.p) + b * w.c.sb + g * w.c.sg;
        u64 y = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = n0 + 2 * i;
            const bool one = on && n < w.N, two = on && n + 1 < w.N;
            const u64 bb = pk(one ? to_f(pb[n]) : 0.f, two ? to_f(pb[n + 1]) : 0.f);
            const u64 cc = pk(one ? to_f(pc[n]) : 0.f, two ? to_f(pc[n + 1]) : 0.f);
            const u64 e = decay_less_one(mul2(splat(s), mul2(a[i], splat(kLog2eF))));
            h[i] = fma2(e, h[i], fma2(splat(s * x), bb, h[i]));
            y = fma2(cc, h[i], y);
        }
        float out = pair_sum(y);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) out += __shfl_xor_sync(0xffffffffu, out, o);
        if (on && n0 == 0) {
            out = fmaf(skip, x, out);
            if (w.gate.p != nullptr) out = gate_with(out, to_f(static_cast<const T *>(w.gate.p)[b * w.gate.sb + d]));
            py[static_cast<long long>(b) * w.D + d] = from_f<T>(out);
        }
        if (w.slots == nullptr) break;
        for (int i = b + 1 + tid; i < w.B; i += 256)
            if (w.slots[i] == slot) {
                atomicMin(&next, i);
                break;
            }
        __syncthreads();
        b = next;
        if (b >= w.B) break;
        __syncthreads();
    }
    if (on) store_states(h, w.out_state + at, n0, w.N, vec);
}

template <typename T, int L>
void launch_step(const SsStep &w, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>((w.D + 256 / L - 1) / (256 / L)) * w.B;
    ss_step_kernel<T, L><<<grid, 256, 0, s>>>(w);
}
template <typename T>
void step_of(const SsStep &w, cudaStream_t s) {
    switch (lanes(w.N)) {
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
