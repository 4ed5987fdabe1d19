// linear_attention.cu -- linear attention with a decay for each head (sm_100a): the sweep of
// linear_attention.cuh for fp32 operands on CUDA cores, the join of time segments, the sum over heads that share
// keys and values, packing for rows that TMA cannot read, and the single-token step.
#include <cuda_bf16.h>

#include "linear_attention.cuh"

namespace pararnn {
namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16(x); }

// Four consecutive elements, n of which exist; VEC: all four, aligned to 16 bytes.
template <bool VEC>
__device__ __forceinline__ float4 load4(const float *p, int n) {
    if (VEC) return *reinterpret_cast<const float4 *>(p);
    return make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
}

__device__ __forceinline__ int row_count(const LaSweep &w, int b) {
    if (w.lengths == nullptr) return w.T;
    const int n = w.lengths[b];
    return n < 0 ? 0 : (n > w.T ? w.T : n);
}

constexpr int kC = 32;     // rows per chunk
constexpr int kThr = 256;

template <int DKP, int DVT>
constexpr int simt_smem_floats() {
    return 2 * kC * (DKP + 4) + 2 * kC * (DVT + 4) + kC * (kC + 4) + DKP * (DVT + 4) + kC + 4 + 2 * kC;
}

// (a, b) += x (u, v): two FMAs in one instruction, for half the issue slots ([5, 2011, 12 x 96 / 80]: 291 -> 270 us)
__device__ __forceinline__ void fma2(float &a, float &b, float x, float u, float v) {
    asm("{.reg .b64 p, q, r; mov.b64 p, {%0, %1}; mov.b64 q, {%2, %2}; mov.b64 r, {%3, %4}; fma.rn.f32x2 p, q, r, p; "
        "mov.b64 {%0, %1}, p;}"
        : "+f"(a), "+f"(b)
        : "f"(x), "f"(u), "f"(v));
}
__device__ __forceinline__ void fma4(float4 &acc, float x, const float4 &y) {
    fma2(acc.x, acc.y, x, y.x, y.y);
    fma2(acc.z, acc.w, x, y.z, y.w);
}
__device__ __forceinline__ float4 *f4(float *p) { return reinterpret_cast<float4 *>(p); }
__device__ __forceinline__ float2 *f2(float *p) { return reinterpret_cast<float2 *>(p); }

// Four rows of a thread's columns j .. j + 3 and, with WIDE, e and e + 1
template <bool WIDE>
struct Piece {
    float4 v[4];
    float2 w[WIDE ? 4 : 1];
};
// acc[u] += sum_d x[u][d] y[d][columns], rows of x and y PX and PY floats apart
template <int PX, int PY, bool WIDE>
__device__ __forceinline__ void product(Piece<WIDE> &acc, float *x, float *y, int j, int e, int depth) {
#pragma unroll 2
    for (int d = 0; d < depth; d += 4) {
        float4 xv[4], yv[4];
        float2 zv[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            xv[u] = *f4(x + u * PX + d);
            yv[u] = *f4(y + (d + u) * PY + j);
            if (WIDE) zv[u] = *f2(y + (d + u) * PY + e);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float f[4] = {xv[u].x, xv[u].y, xv[u].z, xv[u].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                fma4(acc.v[u], f[k], yv[k]);
                if constexpr (WIDE) fma2(acc.w[u].x, acc.w[u].y, f[k], zv[k].x, zv[k].y);
            }
        }
    }
}

struct LaBatch {
    LaSweep w[3];
};

// One CTA: DVT columns of c of one head and one segment, 32 rows at a time, the state in shared memory; fp32 FMAs.
// Warps 0-3 form a S while warps 4-7 form the weighted scores and their product with c; then all update S.  The
// next chunk's rows are loaded into registers before a chunk's arithmetic.  Bound by shared-memory loads (8 of 16
// bytes for 64 FMAs; the data pipe is busy 72 % of the time, FMA issue 35 %); 32 rows, because the scores' share of
// the arithmetic grows with them.
// 8 x 2048 tokens, 16 heads of 128: 750 us, 26 TFLOP/s; five sequences of up to 2011 tokens, 12 heads of 96 and 80:
// 201 us with tiles of 96 columns (before the weights of two rows were read at once 205, and 270 with 64 + 16).
// STATE_ONLY is pass 1 of a split sweep: the segment's own S_out, without a and without outputs.
template <bool VEC, int DKP, int DVT, bool STATE_ONLY>
__global__ void __launch_bounds__(kThr, 2) la_simt_kernel(const __grid_constant__ LaBatch batch) {
    const LaSweep &w = batch.w[blockIdx.z];
    if (blockIdx.x >= w.B * w.H * ((w.dv + DVT - 1) / DVT)) return;  // the grid is the widest sweep's
    constexpr int PK = DKP + 4, PV = DVT + 4, PP = kC + 4;
    constexpr bool WIDE = DVT > 64;
    static_assert(DVT == 64 || DVT == 96, "columns per thread");
    extern __shared__ __align__(16) float sm[];
    float *As = sm, *Bs = As + kC * PK, *Cs = Bs + kC * PK, *Os = Cs + kC * PV, *Ps = Os + kC * PV, *Ss = Ps + kC * PP;
    float *pw = Ss + DKP * PV;  // g^0 .. g^C, and what is left of g^C and of the last chunk's g^n
    float *uw = pw + kC + 4;    // update g^(n - e - j) of row j, of a full chunk and of the last one, zero from n on

    const int tid = threadIdx.x;
    const int n_tile = (w.dv + DVT - 1) / DVT;
    const int bh = blockIdx.x / n_tile, c0 = (blockIdx.x % n_tile) * DVT;
    const int b = bh / w.H, h = bh % w.H, sg = blockIdx.y;
    const int L = row_count(w, b);
    if (STATE_ONLY && sg == (w.reverse ? 0 : w.n_seg - 1)) return;  // nobody starts from its state
    // tokens [t_lo, t_hi) of this segment as logical rows [lo, hi)
    const long long t_lo = static_cast<long long>(sg) * w.seg;
    const int lo_t = t_lo < L ? static_cast<int>(t_lo) : L, hi_t = t_lo + w.seg < L ? static_cast<int>(t_lo + w.seg) : L;
    const int lo = w.reverse ? L - hi_t : lo_t, hi = w.reverse ? L - lo_t : hi_t;
    const int ncol = min(DVT, w.dv - c0);
    const float ld = safe_log_decay(w.log_decay[h]);
    for (int i = tid; i <= kC; i += kThr) pw[i] = decay_pow(ld, i);
    const int n_last = (hi - lo + kC - 1) % kC + 1;
    if (tid >= kThr - 2) pw[kC + 1 + kThr - 1 - tid] = decay_rest(ld, tid == kThr - 1 ? kC : n_last);
    for (int i = tid; i < 2 * kC; i += kThr) {
        const int j = i % kC, n = i < kC ? kC : n_last;
        uw[i] = j < n ? decay_pow(ld, n - w.e - j) * w.update : 0.f;
    }

    // the state this segment starts from
    const long long sbase = static_cast<long long>(bh) * w.dk * w.dv;
    for (int i = tid; i < DKP * DVT; i += kThr) {
        const int d = i / DVT, c = i % DVT;
        float x = 0.f;
        if (!STATE_ONLY && d < w.dk && c < ncol) {
            if (w.n_seg > 1)
                x = w.seg_state[(static_cast<long long>(bh) * w.n_seg + sg) * w.dk * w.dv +
                                static_cast<long long>(d) * w.dv + c0 + c];
            else if (w.s_in != nullptr)
                x = w.s_in[sbase + static_cast<long long>(d) * w.s_i + static_cast<long long>(c0 + c) * w.s_j];
        }
        Ss[d * PV + c] = x;
    }

    const float *pa = static_cast<const float *>(w.a.p) + b * w.a.sb + (h / w.a.group) * w.a.sh;
    const float *pb = static_cast<const float *>(w.b.p) + b * w.b.sb + (h / w.b.group) * w.b.sh;
    const float *pc = static_cast<const float *>(w.c.p) + b * w.c.sb + (h / w.c.group) * w.c.sh + c0;
    float *po = static_cast<float *>(w.out) + (static_cast<long long>(b) * w.T * w.H + h) * w.out_w + c0;
    const long long ost = static_cast<long long>(w.H) * w.out_w;
    const bool rev = w.reverse != 0;
    const int e = w.e;
    const float intra = w.intra, inter = w.inter;

    // this thread's pieces of the next chunk: a, b [C][DKP] and c [C][DVT], zeros outside
    constexpr int NK = kC * DKP / 4 / kThr, NV = kC * DVT / 4 / kThr;
    float4 ra[NK], rb[NK], rc[NV];
    auto fetch = [&](int r0) {
        const int n = min(kC, hi - r0);
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            const int i = tid + k * kThr, r = i / (DKP / 4), d = (i % (DKP / 4)) * 4;
            ra[k] = rb[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < n && d < w.dk) {
                const long long t = rev ? L - 1 - (r0 + r) : r0 + r;
                if (!STATE_ONLY) ra[k] = load4<VEC>(pa + t * w.a.st + d, w.dk - d);
                rb[k] = load4<VEC>(pb + t * w.b.st + d, w.dk - d);
            }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = tid + k * kThr, r = i / (DVT / 4), c = (i % (DVT / 4)) * 4;
            rc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < n && c < ncol) {
                const long long t = rev ? L - 1 - (r0 + r) : r0 + r;
                rc[k] = load4<VEC>(pc + t * w.c.st + c, ncol - c);
            }
        }
    };
    if (lo < hi) fetch(lo);
    for (int r0 = lo; r0 < hi; r0 += kC) {
        const int n = min(kC, hi - r0);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            const int i = tid + k * kThr, at = i / (DKP / 4) * PK + (i % (DKP / 4)) * 4;
            if (!STATE_ONLY) *f4(As + at) = ra[k];
            *f4(Bs + at) = rb[k];
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = tid + k * kThr;
            *f4(Cs + i / (DVT / 4) * PV + (i % (DVT / 4)) * 4) = rc[k];
        }
        __syncthreads();
        if (r0 + kC < hi) fetch(r0 + kC);
        if (!STATE_ONLY) {
            const int t = tid & 127, i0 = (t / 16) * 4, j0 = (t % 16) * 4;  // each half's 128 threads: 4 rows, 4 or 6
            const int e0 = 64 + (t % 16) * 2;                            // columns each
            Piece<WIDE> acc = {};
            if (tid < 128) {
                if (i0 < n) product<PK, PV, WIDE>(acc, As + i0 * PK, Ss, j0, e0, DKP);
            } else {
                // P = (a b^T) weighted, 2 x 4 per thread
                const int p0 = (t / 8) * 2, q0 = t % 8;
                float s[2][4] = {};
                if (p0 < n) {
#pragma unroll 4
                    for (int d = 0; d < DKP; d += 4) {
                        float4 x[2], y[4];
#pragma unroll
                        for (int u = 0; u < 2; ++u) x[u] = *f4(As + (p0 + u) * PK + d);
#pragma unroll
                        for (int u = 0; u < 4; ++u) y[u] = *f4(Bs + (q0 + 8 * u) * PK + d);
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                s[u][q] += x[u].x * y[q].x + x[u].y * y[q].y + x[u].z * y[q].z + x[u].w * y[q].w;
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int i = p0 + u, j = q0 + 8 * q;
                        Ps[i * PP + j] = i >= j ? s[u][q] * pw[i >= j ? i - j : 0] * intra : 0.f;
                    }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (i0 < n) product<PP, PV, WIDE>(acc, Ps + i0 * PP, Cs, j0, e0, i0 + 4);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    *f4(Os + (i0 + u) * PV + j0) = acc.v[u];
                    if constexpr (WIDE) *f2(Os + (i0 + u) * PV + e0) = acc.w[u];
                }
            }
            __syncthreads();
            if (tid < 128) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (i0 + u < n) {
                        const float g = pw[min(i0 + u + e, kC)] * inter;
                        const float4 y = *f4(Os + (i0 + u) * PV + j0);
                        const long long tok = rev ? L - 1 - (r0 + i0 + u) : r0 + i0 + u;
                        float *o = po + tok * ost;
                        const float4 x = make_float4(fmaf(g, acc.v[u].x, y.x), fmaf(g, acc.v[u].y, y.y),
                                                     fmaf(g, acc.v[u].z, y.z), fmaf(g, acc.v[u].w, y.w));
                        if (VEC) {  // widths are multiples of 4
                            if (j0 < ncol) *f4(o + j0) = x;
                        } else {
                            const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                if (j0 + q < ncol) o[j0 + q] = f[q];
                        }
                        if constexpr (WIDE) {
                            const float2 z = *f2(Os + (i0 + u) * PV + e0);
                            const float2 v = make_float2(fmaf(g, acc.w[u].x, z.x), fmaf(g, acc.w[u].y, z.y));
                            if (VEC) {
                                if (e0 < ncol) *f2(o + e0) = v;
                            } else {
                                if (e0 < ncol) o[e0] = v.x;
                                if (e0 + 1 < ncol) o[e0 + 1] = v.y;
                            }
                        }
                    }
            }
        }
        {  // S = g^n S + update sum_j g^(n-e-j) b_j c_j^T: DKP / 32 x DVT / 8 per thread; the chunk's sum by itself, so that
           // a state of many chunks is rounded once each and not once a token
            constexpr int RD = DKP / 32, CD = DVT / 32;
            const int d0 = (tid / 8) * RD, j0 = (tid % 8) * 4;
            float4 acc[RD][CD] = {};
            const float gn = pw[n], gn_rest = pw[n < kC ? kC + 2 : kC + 1];
            const float *wj = uw + (n < kC ? kC : 0);
#pragma unroll 2
            for (int r = 0; r < n; r += 2) {  // rows from n on are zero
                const float2 f = *reinterpret_cast<const float2 *>(wj + r);
                const float g[2] = {f.x, f.y};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int j = r + k;
                    float x[RD];
                    if constexpr (RD == 4) {
                        const float4 v = *f4(Bs + j * PK + d0);
                        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
                    } else {
#pragma unroll
                        for (int u = 0; u < RD; ++u) x[u] = Bs[j * PK + d0 + u];
                    }
                    float4 y[CD];
#pragma unroll
                    for (int q = 0; q < CD; ++q) y[q] = *f4(Cs + j * PV + j0 + 32 * q);
#pragma unroll
                    for (int u = 0; u < RD; ++u)
#pragma unroll
                        for (int q = 0; q < CD; ++q) fma4(acc[u][q], x[u] * g[k], y[q]);
                }
            }
#pragma unroll
            for (int u = 0; u < RD; ++u)
#pragma unroll
                for (int q = 0; q < CD; ++q) {
                    float4 *const at = f4(Ss + (d0 + u) * PV + j0 + 32 * q);
                    const float4 s = *at;
                    fma4(acc[u][q], gn_rest, s);
                    fma4(acc[u][q], gn, s);
                    *at = acc[u][q];
                }
        }
    }
    __syncthreads();
    if (STATE_ONLY) {
        for (int i = tid; i < w.dk * ncol; i += kThr) {
            const int d = i / ncol, c = i % ncol;
            w.seg_state[(static_cast<long long>(bh) * w.n_seg + sg) * w.dk * w.dv +
                        static_cast<long long>(d) * w.dv + c0 + c] = Ss[d * PV + c];
        }
        return;
    }
    const int last = L > 0 && !w.reverse ? (L - 1) / w.seg : 0;  // the segment that holds the last logical row
    if (w.s_out != nullptr && sg == last)
        for (int i = tid; i < w.dk * ncol; i += kThr) {
            const int d = w.s_j == 1 ? i / ncol : i % w.dk, c = w.s_j == 1 ? i % ncol : i / w.dk;
            w.s_out[sbase + static_cast<long long>(d) * w.s_i + static_cast<long long>(c0 + c) * w.s_j] =
                Ss[d * PV + c];
        }
    // outputs behind the sequence's length are zero
    const long long z_hi = t_lo + w.seg < w.T ? t_lo + w.seg : w.T;
    for (long long t = (t_lo > L ? t_lo : L); t < z_hi; ++t)
        for (int c = tid; c < ncol; c += kThr) po[t * ost + c] = 0.f;
}

// Join of a split sweep, in place: seg_state[s] (segment s's own state) becomes the state segment s starts from.
// A thread per element; the segments' own states are loaded eight at a time, ahead of the recurrence.
__global__ void __launch_bounds__(256) la_join_kernel(const LaSweep w) {
    constexpr int KB = 8;
    const int n = w.dk * w.dv;
    const int per = (n + 255) / 256;  // CTAs per head
    const int bh = blockIdx.x / per, i = (blockIdx.x % per) * 256 + threadIdx.x;
    const float ld = safe_log_decay(w.log_decay[bh % w.H]);
    const int L = row_count(w, bh / w.H);
    // the segment with the sequence's end, where it is not full
    const int q_part = L / w.seg;
    __shared__ float rest[2];  // of a full segment's weight and of that one's
    if (threadIdx.x < 2) rest[threadIdx.x] = decay_rest(ld, threadIdx.x == 0 ? w.seg : L - q_part * w.seg);
    __syncthreads();
    if (i >= n) return;
    float *p = w.seg_state + static_cast<long long>(bh) * w.n_seg * n + i;
    float s = w.s_in == nullptr ? 0.f : w.s_in[static_cast<long long>(bh) * n + (i / w.dv) * w.s_i + (i % w.dv) * w.s_j];
    const float g_full = decay_pow(ld, w.seg);
    const float g_part = decay_pow(ld, L - q_part * w.seg);
    const int first = w.reverse ? w.n_seg - 1 : 0, dir = w.reverse ? -1 : 1;
    for (int k0 = 0; k0 < w.n_seg; k0 += KB) {
        float own[KB];
#pragma unroll
        for (int k = 0; k < KB; ++k)  // the last one's own state is not wanted
            own[k] = k0 + k + 1 < w.n_seg ? p[static_cast<long long>(first + dir * (k0 + k)) * n] : 0.f;
#pragma unroll
        for (int k = 0; k < KB; ++k)
            if (k0 + k < w.n_seg) {
                const int q = first + dir * (k0 + k);
                p[static_cast<long long>(q) * n] = s;
                if (q <= q_part) s = fmaf(q < q_part ? g_full : g_part, s, fmaf(rest[q < q_part ? 0 : 1], s, own[k]));
            }
    }
}

}  // namespace

cudaError_t launch_la_join(const LaSweep &w, cudaStream_t s) {
    la_join_kernel<<<static_cast<unsigned>(w.B) * w.H * ((w.dk * w.dv + 255) / 256), 256, 0, s>>>(w);
    return cudaGetLastError();
}

namespace {

template <bool VEC, int DKP, int DVT>
cudaError_t launch_simt(const LaBatch &t, int n, cudaStream_t s) {
    const int smem = simt_smem_floats<DKP, DVT>() * 4;
    unsigned tiles = 0;
    for (int i = 0; i < n; ++i) tiles = max(tiles, static_cast<unsigned>((t.w[i].dv + DVT - 1) / DVT));
    const LaSweep &w = t.w[0];
    const dim3 grid(static_cast<unsigned>(w.B) * w.H * tiles, w.n_seg, n);
    cudaError_t e;
    if (w.n_seg > 1) {
        auto k1 = la_simt_kernel<VEC, DKP, DVT, true>;
        if ((e = cudaFuncSetAttribute(k1, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
        k1<<<grid, kThr, smem, s>>>(t);
        for (int i = 0; i < n; ++i)
            if ((e = launch_la_join(t.w[i], s)) != cudaSuccess) return e;
    }
    auto k = la_simt_kernel<VEC, DKP, DVT, false>;
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    k<<<grid, kThr, smem, s>>>(t);
    return cudaGetLastError();
}

// width of a and b that the kernel is compiled for
int simt_width(int dk) { return dk <= 32 ? 32 : dk <= 64 ? 64 : dk <= 96 ? 96 : 128; }
// columns of c per CTA: 96 for 65 to 96 of them, where the state leaves shared memory for two CTAs per SM
int simt_tile(int dk, int dv) { return dk <= 96 && dv > 64 && dv <= 96 ? 96 : 64; }

bool rows_vec4(const LaRows &x) {
    return reinterpret_cast<uintptr_t>(x.p) % 16 == 0 && x.sb % 4 == 0 && x.st % 4 == 0 && x.sh % 4 == 0;
}
bool simt_vec(const LaSweep &w) {
    return w.dk % 4 == 0 && w.dv % 4 == 0 && w.out_w % 4 == 0 && rows_vec4(w.a) && rows_vec4(w.b) && rows_vec4(w.c);
}

template <bool VEC>
cudaError_t pick_width(const LaBatch &t, int n, cudaStream_t s) {
    const bool wide = simt_tile(t.w[0].dk, t.w[0].dv) == 96;
    switch (simt_width(t.w[0].dk)) {
        case 32: return wide ? launch_simt<VEC, 32, 96>(t, n, s) : launch_simt<VEC, 32, 64>(t, n, s);
        case 64: return wide ? launch_simt<VEC, 64, 96>(t, n, s) : launch_simt<VEC, 64, 64>(t, n, s);
        case 96: return wide ? launch_simt<VEC, 96, 96>(t, n, s) : launch_simt<VEC, 96, 64>(t, n, s);
        default: return launch_simt<VEC, 128, 64>(t, n, s);
    }
}

// n <= 3 sweeps in one launch
cudaError_t launch_la_simt(const LaSweep *w, int n, cudaStream_t s) {
    LaBatch t{};
    for (int i = 0; i < n; ++i) t.w[i] = w[i];
    return simt_vec(w[0]) ? pick_width<true>(t, n, s) : pick_width<false>(t, n, s);
}
bool simt_together(const LaSweep &x, const LaSweep &y) {
    return simt_width(x.dk) == simt_width(y.dk) && simt_tile(x.dk, x.dv) == simt_tile(y.dk, y.dv) && simt_vec(x) == simt_vec(y) && x.n_seg == y.n_seg && x.seg == y.seg;
}

}  // namespace

LaPlan la_plan(int B, int T, int H, int dk, int dv, int dtype, int sweeps, bool ragged) {
    const long long heads = static_cast<long long>(B) * H * sweeps;
    long long want, most;
    int unit;
    if (dtype == PARARNN_BF16) {
        // one CTA per SM: as many segments as fill the 148 SMs once.  A split costs about 1.6 times a segment's chunks,
        // since pass 1 takes 0.6 of pass 2's time, and its two more launches as much as 6 chunks, or 9 with three joins
        // in a row; so two segments are no gain, nor are short sequences (unsplit against split, forward 512 tokens of
        // 8 heads of 64 16.4 / 22.5 us, 1024 24.6 / 24.6, 2048 41 / 26; backward 1024 27 / 31, 2048 43 / 35; backward of
        // 16 heads of 128, 2048 tokens 68 / 78, 4096 121 / 107)
        const int chunks = (T + 127) / 128;
        want = 148 / heads;
        if (want > chunks) want = chunks;
        if (want < 3 || 8 * ((chunks + want - 1) / want) + 5 * (sweeps == 1 ? 6 : 9) >= 5 * chunks) want = 1;
        most = chunks;
        unit = 128;
    } else {
        // two CTAs per SM, filled once, in segments of at least 64 rows ([1, 512, 4 x 64] forward 47 us with at least
        // 128, 35 with 64, 31 with 32; ragged [3, 517, 6 x 48 / 64] backward 90, 70, 74); 1.5 times that many CTAs
        // where lengths may differ, so that short sequences leave room.  On eight ragged shapes with two sets of lengths
        // each (2 to 16 sequences of up to 700 to 8192 tokens, 4 to 24 heads of 64 to 128) the best count of segments
        // varies with the lengths, as the longest sequences' segments fall on SMs; 444 CTAs are 1.06 times the best one's
        // time in the geometric mean, 1.27 at most, 296 are 1.15 and 1.43, 592 are 1.11 and 1.31
        const long long ctas = heads * ((dv + simt_tile(dk, dv) - 1) / simt_tile(dk, dv));
        want = ragged ? (444 + ctas - 1) / ctas : 296 / ctas;
        most = T / 64;
        unit = kC;
    }
    if (want > most) want = most;
    if (want > 512) want = 512;
    if (want < 2) return {1, T};
    int seg = static_cast<int>((T + want - 1) / want);
    seg = (seg + unit - 1) / unit * unit;
    return {(T + seg - 1) / seg, seg};
}

cudaError_t launch_la_sweeps(const LaSweep *w, int n, cudaStream_t s) {
    for (int i = 0; i < n;) {
        int k = 1;
        cudaError_t e;
        if (w[i].dtype == PARARNN_BF16) {
            while (i + k < n && la_tc_together(w[i], w[i + k])) ++k;
            e = launch_la_tc(w + i, k, s);
        } else {
            while (i + k < n && simt_together(w[i], w[i + k])) ++k;
            e = launch_la_simt(w + i, k, s);
        }
        if (e != cudaSuccess) return e;
        i += k;
    }
    return cudaSuccess;
}

// ---- packing ------------------------------------------------------------------------------------------------

namespace {

// bf16 rows from and to a dense [B, T, heads, wp] (wp: width rounded up to 8), 8 columns per thread
__global__ void la_pack_kernel(const LaRows src, uint4 *__restrict__ dst, int T, int heads, int width, int wp,
                               long long n) {
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<long long>(gridDim.x) * blockDim.x) {
        const int c = static_cast<int>(i % (wp / 8)) * 8;
        const long long row = i / (wp / 8);
        const int h = static_cast<int>(row % heads);
        const long long t = row / heads % T, b = row / heads / T;
        const unsigned short *p =
            static_cast<const unsigned short *>(src.p) + b * src.sb + t * src.st + h * src.sh + c;
        unsigned u[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (c + k < width) u[k >> 1] |= static_cast<unsigned>(p[k]) << (16 * (k & 1));
        dst[i] = make_uint4(u[0], u[1], u[2], u[3]);
    }
}
__global__ void la_unpack_kernel(const uint4 *__restrict__ src, unsigned short *__restrict__ dst, int width, int wp,
                                 long long n) {
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<long long>(gridDim.x) * blockDim.x) {
        const int c = static_cast<int>(i % (wp / 8)) * 8;
        unsigned short *p = dst + i / (wp / 8) * width + c;
        const uint4 x = src[i];
        const unsigned u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (c + k < width) p[k] = static_cast<unsigned short>(u[k >> 1] >> (16 * (k & 1)));
    }
}
unsigned pack_grid(long long n) { return static_cast<unsigned>(n / 256 + 1 < 148 * 16 ? n / 256 + 1 : 148 * 16); }

}  // namespace

cudaError_t launch_la_pack(const LaRows &src, void *dst, int B, int T, int heads, int width, cudaStream_t s) {
    const int wp = (width + 7) / 8 * 8;
    const long long n = static_cast<long long>(B) * T * heads * (wp / 8);
    la_pack_kernel<<<pack_grid(n), 256, 0, s>>>(src, static_cast<uint4 *>(dst), T, heads, width, wp, n);
    return cudaGetLastError();
}

cudaError_t launch_la_unpack(const void *src, void *dst, long long rows, int width, cudaStream_t s) {
    const int wp = (width + 7) / 8 * 8;
    const long long n = rows * (wp / 8);
    la_unpack_kernel<<<pack_grid(n), 256, 0, s>>>(static_cast<const uint4 *>(src), static_cast<unsigned short *>(dst), width,
                                                  wp, n);
    return cudaGetLastError();
}

// ---- sums over the heads that share a key/value head --------------------------------------------------------

namespace {

// out[row, u, :d] = sum over the `per` heads of group u of part[row, u * per + i, :d], in head order; rows of part are
// dp wide
template <typename TO>
__global__ void la_group_sum_kernel(const float *__restrict__ part, TO *__restrict__ out, long long rows, int Hkv,
                                    int per, int d, int dp) {
    const long long n = rows * Hkv * d;
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<long long>(gridDim.x) * blockDim.x) {
        const long long ru = i / d;  // row * Hkv + u
        const int c = static_cast<int>(i % d);
        const float *p = part + ru * per * dp + c;
        float s = 0.f;
        for (int q = 0; q < per; ++q) s += p[static_cast<long long>(q) * dp];
        out[i] = from_f<TO>(s);
    }
}

}  // namespace

cudaError_t launch_la_group_sum(const float *part, void *out, int dtype, long long rows, int Hkv, int per, int d,
                                int dp, cudaStream_t s) {
    const long long n = rows * Hkv * d;
    const unsigned grid = static_cast<unsigned>(n / 256 + 1 < 148 * 16 ? n / 256 + 1 : 148 * 16);
    if (dtype == PARARNN_F32)
        la_group_sum_kernel<<<grid, 256, 0, s>>>(part, static_cast<float *>(out), rows, Hkv, per, d, dp);
    else
        la_group_sum_kernel<<<grid, 256, 0, s>>>(part, static_cast<__nv_bfloat16 *>(out), rows, Hkv, per, d, dp);
    return cudaGetLastError();
}

// ---- one token per sequence ---------------------------------------------------------------------------------

namespace {

// One CTA per row and head: S = g S + k v^T, out = scale S^T q.  Thread (ty, tx) holds VW consecutive columns of
// every NY-th row of S; the column sums meet in shared memory.  Rows of the batch that name the same slot are
// taken in row order by the first one's CTA: tokens that follow each other.  Bound by HBM, as each state is read and
// written once: 256 rows, 16 heads of 128 x 128 take 89 us, 541 MB at 0.93 of a copy's rate.  Each CTA reads all slots
// once, without a workspace: 108 against 103 us without slots on those 256 rows from cold caches, 1459 against 1291 on 4096,
// 7673 against 5091 on 16384.
template <typename TI, int VW>
__global__ void __launch_bounds__(256) la_step_kernel(const LaStep w) {
    __shared__ float qs[128], ks[128], part[256 * VW];
    __shared__ int next;
    const int tid = threadIdx.x;
    const int h = blockIdx.x % w.H;
    int b = blockIdx.x / w.H;
    const int NX = (w.dv + VW - 1) / VW, NY = blockDim.x / NX;
    const int tx = tid % NX, ty = tid / NX;
    TI *po = static_cast<TI *>(w.out);
    const int slot = w.slots == nullptr ? b : w.slots[b];
    if (slot < 0 || slot >= w.n_slots) {  // no state behind this row
        for (int c = tid; c < w.dv; c += blockDim.x)
            po[(static_cast<long long>(b) * w.H + h) * w.dv + c] = from_f<TI>(0.f);
        return;
    }
    if (w.slots != nullptr) {
        int earlier = 0;
        for (int i = tid; i < b; i += blockDim.x) earlier |= w.slots[i] == slot;
        if (__syncthreads_or(earlier)) return;
    }
    // g and what rounding leaves of it: one fp32 would be another decay, taken at every token (4096 tokens with a memory of
    // 1e6: 2e-4 of the state).  Below e^-1/2 a state is forgotten before that counts.
    const float ld = safe_log_decay(w.log_decay[h]), below = ld > -0.5f ? expm1f(ld) : 0.f;
    const float g = ld > -0.5f ? 1.f + below : expf(ld), g_rest = ld > -0.5f ? below - (g - 1.f) : 0.f;
    const long long base = (static_cast<long long>(slot) * w.H + h) * w.dk * w.dv;
    const float *src = w.state + base;
    float *dst = w.out_state + base;
    while (true) {
        const TI *q = static_cast<const TI *>(w.q.p) + b * w.q.sb + (h / w.q.group) * w.q.sh;
        const TI *k = static_cast<const TI *>(w.k.p) + b * w.k.sb + (h / w.k.group) * w.k.sh;
        const TI *v = static_cast<const TI *>(w.v.p) + b * w.v.sb + (h / w.v.group) * w.v.sh;
        for (int d = tid; d < w.dk; d += blockDim.x) {
            qs[d] = to_f(q[d]) * w.scale;
            ks[d] = to_f(k[d]);
        }
        if (tid == 0) next = w.B;
        __syncthreads();
        float acc[VW] = {};
        if (ty < NY) {
            float vv[VW];
#pragma unroll
            for (int u = 0; u < VW; ++u) vv[u] = tx * VW + u < w.dv ? to_f(v[tx * VW + u]) : 0.f;
            constexpr int RB = VW == 4 ? 8 : 16;  // rows of S in flight
            for (int d0 = ty; d0 < w.dk; d0 += RB * NY) {
                float s[RB][VW];
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    const int d = d0 + r * NY;
                    if (d >= w.dk) break;
                    const float *p = src + d * w.dv + tx * VW;
                    if constexpr (VW == 4) {
                        const float4 x = __ldcs(reinterpret_cast<const float4 *>(p));
                        s[r][0] = x.x, s[r][1] = x.y, s[r][2] = x.z, s[r][3] = x.w;
                    } else {
                        s[r][0] = *p;
                    }
                }
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    const int d = d0 + r * NY;
                    if (d >= w.dk) break;
#pragma unroll
                    for (int u = 0; u < VW; ++u) {
                        s[r][u] = fmaf(g, s[r][u], fmaf(ks[d], vv[u], g_rest * s[r][u]));
                        acc[u] = fmaf(qs[d], s[r][u], acc[u]);
                    }
                    float *p = dst + d * w.dv + tx * VW;
                    if constexpr (VW == 4)
                        __stcs(reinterpret_cast<float4 *>(p), make_float4(s[r][0], s[r][1], s[r][2], s[r][3]));
                    else
                        *p = s[r][0];
                }
            }
#pragma unroll
            for (int u = 0; u < VW; ++u) part[ty * NX * VW + tx * VW + u] = acc[u];
        }
        if (w.slots != nullptr)
            for (int i = b + 1 + tid; i < w.B; i += blockDim.x)
                if (w.slots[i] == slot) {
                    atomicMin(&next, i);
                    break;
                }
        __syncthreads();
        for (int c = tid; c < w.dv; c += blockDim.x) {
            float s = 0.f;
            for (int y = 0; y < NY; ++y) s += part[y * NX * VW + c];
            po[(static_cast<long long>(b) * w.H + h) * w.dv + c] = from_f<TI>(s);
        }
        b = next;
        if (b >= w.B) return;
        src = dst;  // each thread reads back what it wrote itself
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_la_step(const LaStep &w, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(w.B) * w.H;
    const bool vec = w.dv % 4 == 0;
    if (w.dtype == PARARNN_F32) {
        if (vec) la_step_kernel<float, 4><<<grid, 256, 0, s>>>(w);
        else la_step_kernel<float, 1><<<grid, 256, 0, s>>>(w);
    } else {
        if (vec) la_step_kernel<__nv_bfloat16, 4><<<grid, 256, 0, s>>>(w);
        else la_step_kernel<__nv_bfloat16, 1><<<grid, 256, 0, s>>>(w);
    }
    return cudaGetLastError();
}

}  // namespace pararnn
