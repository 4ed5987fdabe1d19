// linear_attention_tc.cu -- the sweep of linear_attention.cuh for bf16 operands on the 5th-generation tensor
// cores (tcgen05, sm_100a).
//
// One CTA carries one head's state (dv columns of it) through one segment of time, 128 rows at a time:
//   scores = a b^T                      [128 x 128]  operands in shared memory
//   out    = g^(i+e) (a S)              [128 x DV]   S as a bf16 copy in shared memory
//   out   += (scores * g^(i-j)) c       [128 x DV]   weighted scores rounded to bf16 in TMEM as the A operand
//   dS^T   = (g^(n-e-j) c)^T b          [DV x DK]    weighted c in TMEM as the A operand
//   S      = g^n S + dS                 in registers, fp32
// A bf16 product is exact in fp32, so the only roundings below fp32 are those of the weighted scores and of S's
// copy, each 2^-9 relative as the output's own.  The weighted c is split into three bf16 terms (24 bits), so the
// state's products are exact to fp32; they are summed smallest term first.
//
// Warps: 0-3 output rows (thread = row: weigh scores, scale, store), 4-11 state (lane quarter = columns of c,
// two warpgroups share the width of b and the rows to be split), 12 issues the products, 13-15 copy the next
// chunk's tiles with cp.async (zero-filled outside, 128-byte swizzle) into the other of two stages.  Every wait
// is bounded; a wait that runs out marks this CTA's results NaN.
#include <cuda_bf16.h>

#include "linear_attention.cuh"
#include "tc_utils.cuh"

namespace pararnn {
namespace {
using namespace tc;

constexpr int kC = 128;       // rows per chunk
constexpr int kThreads = 512;
constexpr int kLoaders = 96;
constexpr int kPanel = kC * 128;  // bytes of a [128 rows][64 bf16] panel

template <int DK, int DV>
struct Lay {
    static constexpr int A = 0, B = A + DK / 64 * kPanel, C = B + DK / 64 * kPanel;
    static constexpr int STAGE = C + DV / 64 * kPanel;
    static constexpr int SS = 2 * STAGE;                    // bf16 S: [DV rows][DK], K-major panels
    static constexpr int TAB = SS + DK / 64 * DV * 128;     // floats: powers 256, score weights 160
    static constexpr int BARS = TAB + (256 + 160) * 4;
    static constexpr int BYTES = BARS + 256 + 1024;
    // TMEM columns: scores 0-127, of which 0-63 become the weighted scores; out; three terms of c; dS in one or
    // two 64-column halves, the first in the half of the scores that is free by then
    static constexpr int T_P = 0, T_O = 128, T_V = 256, T_D0 = DK == 128 ? 64 : 448, T_D1 = 448;
    static constexpr int STATE_WARPS = 2 * (DV / 32);
    static_assert(BYTES <= 227 * 1024, "shared memory");
};

struct Bars {
    unsigned long long full[2], empty[2], scores, inter, p, v, ss, out, ds, out_read, ds_read, drain;
    unsigned tmem;
    int err;
};

__device__ __forceinline__ void arrive(unsigned bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void commit(unsigned bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// N-major operand (rows of the contraction, 64 columns per 128-byte swizzled panel): 8-row groups 1024 bytes apart
// (SBO), panels kPanel apart (LBO).
__device__ __forceinline__ unsigned long long nmajor_desc(unsigned addr) {
    unsigned long long d = 0;
    d |= static_cast<unsigned long long>((addr >> 4) & 0x3fffu);
    d |= static_cast<unsigned long long>(kPanel >> 4) << 16;
    d |= static_cast<unsigned long long>(1024u >> 4) << 32;
    d |= static_cast<unsigned long long>(1u) << 46;
    d |= static_cast<unsigned long long>(2u) << 61;
    return d;
}
constexpr unsigned kNMajorB = 1u << 16;  // instruction descriptor: B is N-major

__device__ __forceinline__ void mma_ss(unsigned d, unsigned long long a, unsigned long long b, unsigned idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u));
}
__device__ __forceinline__ void mma_ts(unsigned d, unsigned a, unsigned long long b, unsigned idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u));
}

__device__ __forceinline__ void tmem_ld32(unsigned addr, float (&v)[32]) {
    unsigned *r = reinterpret_cast<unsigned *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
        "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st32(unsigned addr, const float (&v)[32]) {
    const unsigned *r = reinterpret_cast<const unsigned *>(v);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
        "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]));
}
__device__ __forceinline__ void tmem_st16(unsigned addr, const unsigned (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ unsigned pack(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const unsigned *>(&p);
}
__device__ __forceinline__ float lo_of(unsigned u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_of(unsigned u) { return __uint_as_float(u & 0xffff0000u); }

// One tile: row r of the chunk is token t0 + dir * r; rows >= n and columns >= width are zero.
template <int PANELS>
__device__ __forceinline__ void copy_tile(unsigned dst, const __nv_bfloat16 *src, long long st, long long t0, int dir,
                                          int n, int width, bool vec, int lt) {
    constexpr int CH = PANELS * 8, RP = kLoaders / CH;
    const int c = lt % CH;
    const int room = width - c * 8;  // elements of this 16-byte piece that exist
    const int bytes = room >= 8 ? 16 : (room > 0 ? room * 2 : 0);
    for (int r = lt / CH; r < kC; r += RP) {
        const unsigned at = dst + (c >> 3) * kPanel + r * 128 + (((c & 7) ^ (r & 7)) << 4);
        const __nv_bfloat16 *p = src + (t0 + static_cast<long long>(dir) * r) * st + c * 8;
        if (vec) {
            const int sz = r < n ? bytes : 0;
            if (sz == 0) p = src;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(p), "r"(sz) : "memory");
        } else {
            unsigned u[4] = {0u, 0u, 0u, 0u};
            if (r < n) {
                const unsigned short *q = reinterpret_cast<const unsigned short *>(p);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < room) u[i >> 1] |= static_cast<unsigned>(q[i]) << (16 * (i & 1));
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3])
                         : "memory");
        }
    }
}

template <typename TO>
__device__ __forceinline__ void store32(TO *p, const float (&v)[32], int room, bool vec);
template <>
__device__ __forceinline__ void store32<__nv_bfloat16>(__nv_bfloat16 *p, const float (&v)[32], int room, bool vec) {
    if (vec && room >= 32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4 *>(p + 8 * i) =
                make_uint4(pack(v[8 * i], v[8 * i + 1]), pack(v[8 * i + 2], v[8 * i + 3]),
                           pack(v[8 * i + 4], v[8 * i + 5]), pack(v[8 * i + 6], v[8 * i + 7]));
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < room) p[i] = __float2bfloat16(v[i]);
    }
}
template <>
__device__ __forceinline__ void store32<float>(float *p, const float (&v)[32], int room, bool vec) {
    if (vec && room >= 32) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4 *>(p + 4 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < room) p[i] = v[i];
    }
}

template <typename TO, int DK, int DV, bool STATE_ONLY>
__global__ void __launch_bounds__(kThreads, 1) la_tc_kernel(const __grid_constant__ LaSweep w) {
    using Y = Lay<DK, DV>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                            ~static_cast<uintptr_t>(1023));
    const unsigned sm = smem_u32(smem);
    float *rp = reinterpret_cast<float *>(smem + Y::TAB);  // [256]: g^(128 - x), 0 behind x = 128
    float *sw = rp + 256 + 32;                             // [-32 .. 127]: intra g^x, 0 below x = 0
    Bars *bars = reinterpret_cast<Bars *>(smem + Y::BARS);
    volatile int *err = &bars->err;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int n_tile = (w.dv + DV - 1) / DV;
    const int bh = blockIdx.x / n_tile, c0 = (blockIdx.x % n_tile) * DV;
    const int b = bh / w.H, h = bh % w.H, sg = blockIdx.y;
    int L = w.T;
    if (w.lengths != nullptr) L = min(max(w.lengths[b], 0), w.T);
    const long long r_lo = static_cast<long long>(sg) * w.seg;
    const int lo = r_lo < L ? static_cast<int>(r_lo) : L;
    const int hi = r_lo + w.seg < L ? static_cast<int>(r_lo + w.seg) : L;
    const int chunks = (hi - lo + kC - 1) / kC;
    const int ncol = min(DV, w.dv - c0);

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&bars->full[s]), kLoaders / 32);
            mbar_init(smem_u32(&bars->empty[s]), 1);
        }
        mbar_init(smem_u32(&bars->scores), 1);
        mbar_init(smem_u32(&bars->inter), 1);
        mbar_init(smem_u32(&bars->out), 1);
        mbar_init(smem_u32(&bars->ds), 1);
        mbar_init(smem_u32(&bars->drain), 1);
        mbar_init(smem_u32(&bars->p), 4);
        mbar_init(smem_u32(&bars->out_read), 4);
        mbar_init(smem_u32(&bars->v), Y::STATE_WARPS);
        mbar_init(smem_u32(&bars->ss), Y::STATE_WARPS);
        mbar_init(smem_u32(&bars->ds_read), Y::STATE_WARPS);
        bars->err = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    {
        // exp(n * -1e4) is 0 for n >= 1 and 1 for n = 0, as g = 0 wants it
        const double ld = fmaxf(w.log_decay[h], -1e4f);
        if (tid < 256) rp[tid] = tid <= 128 ? expf(static_cast<float>(ld * (128 - tid))) : 0.f;
        else if (tid < 256 + 160) sw[tid - 288] = tid >= 288 ? expf(static_cast<float>(ld * (tid - 288))) * w.intra : 0.f;
    }
    fence_before();
    __syncthreads();
    fence_after();
    const unsigned tm = bars->tmem;

    if (warp < 4) {
        // ---- output rows: thread = row of the chunk
        if (!STATE_ONLY) {
            const int row = tid;
            const unsigned tl = tm + (static_cast<unsigned>(warp * 32) << 16);
            const float f = rp[128 - row - w.e] * w.inter;
            TO *po = static_cast<TO *>(w.out) + (static_cast<long long>(b) * w.T * w.H + h) * w.dv + c0;
            const long long ost = static_cast<long long>(w.H) * w.dv;
            const bool vec = w.dv % 8 == 0;
            for (int c = 0; c < chunks; ++c) {
                const unsigned ph = c & 1;
                const int r = lo + c * kC + row;
                if (!mbar_wait(smem_u32(&bars->scores), ph, err)) break;
                fence_after();
#pragma unroll 1
                for (int jb = 0; jb < 4; ++jb) {
                    unsigned u[16] = {};
                    if (jb <= warp) {  // columns behind this warp's last row are zero
                        float v[32];
                        tmem_ld32(tl + Y::T_P + jb * 32, v);
                        const float *s = sw + row - jb * 32;
#pragma unroll
                        for (int j = 0; j < 16; ++j) u[j] = pack(v[2 * j] * s[-2 * j], v[2 * j + 1] * s[-2 * j - 1]);
                    }
                    tmem_st16(tl + Y::T_P + jb * 16, u);
                }
                if (!mbar_wait(smem_u32(&bars->inter), ph, err)) break;
                fence_after();
#pragma unroll 1
                for (int cb = 0; cb < DV; cb += 32) {
                    float v[32];
                    tmem_ld32(tl + Y::T_O + cb, v);
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] *= f;
                    tmem_st32(tl + Y::T_O + cb, v);
                }
                tmem_st_wait();
                fence_before();
                __syncwarp();
                if (lane == 0) arrive(smem_u32(&bars->p));
                if (!mbar_wait(smem_u32(&bars->out), ph, err)) break;
                fence_after();
                const long long t = w.reverse ? L - 1 - r : r;
#pragma unroll 1
                for (int cb = 0; cb < DV; cb += 32) {
                    float v[32];
                    tmem_ld32(tl + Y::T_O + cb, v);
                    if (cb == DV - 32) {
                        fence_before();
                        __syncwarp();
                        if (lane == 0) arrive(smem_u32(&bars->out_read));
                    }
                    if (r < hi && cb < ncol) store32<TO>(po + t * ost + cb, v, ncol - cb, vec);
                }
            }
        }
    } else if (warp < 12) {
        // ---- state: lane of TMEM = column of c, half = half of b's width and of the chunk's rows
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        if (quarter * 32 < DV) {
            constexpr int KH = DK / 2;
            const int d = quarter * 32 + lane;
            const unsigned tl = tm + (static_cast<unsigned>(quarter * 32) << 16);
            const unsigned t_ds = tl + (DK == 128 ? (half ? Y::T_D1 : Y::T_D0) : Y::T_D1 + half * KH);
            float S[KH];
            {
                const bool have = d < ncol && (w.n_seg > 1 ? !STATE_ONLY : w.s_in != nullptr);
                const float *p = w.n_seg > 1
                                     ? w.seg_state + (static_cast<long long>(bh) * w.n_seg + sg) * w.dk * w.dv + c0 + d
                                     : w.s_in + static_cast<long long>(bh) * w.dk * w.dv +
                                           static_cast<long long>(c0 + d) * w.s_j;
                const int si = w.n_seg > 1 ? w.dv : w.s_i;
#pragma unroll
                for (int k = 0; k < KH; ++k) {
                    const int kk = half * KH + k;
                    S[k] = have && kk < w.dk ? p[static_cast<long long>(kk) * si] : 0.f;
                }
            }
            // S's bf16 copy: row d, columns half * KH ..
            auto publish = [&]() {
#pragma unroll
                for (int k = 0; k < KH; k += 8) {
                    const int kk = half * KH + k;
                    const unsigned at = sm + Y::SS + (kk >> 6) * (DV * 128) + d * 128 + ((((kk & 63) >> 3) ^ (d & 7)) << 4);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(pack(S[k], S[k + 1])),
                                 "r"(pack(S[k + 2], S[k + 3])), "r"(pack(S[k + 4], S[k + 5])),
                                 "r"(pack(S[k + 6], S[k + 7]))
                                 : "memory");
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) arrive(smem_u32(&bars->ss));
            };
            if (!STATE_ONLY) publish();
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1, n = min(kC, hi - lo - c * kC);
                const unsigned ph = c & 1;
                if (!mbar_wait(smem_u32(&bars->full[st]), (c >> 1) & 1, err)) break;
                const unsigned char *cp = smem + st * Y::STAGE + Y::C + (d >> 6) * kPanel + (d & 7) * 2;
                const int dc = (d & 63) >> 3;
                const float *cw = rp + 128 - n + w.e;  // g^(n - e - j); rows j >= n are zero
#pragma unroll 1
                for (int jb = half * 64; jb < half * 64 + 64; jb += 32) {
                    unsigned u0[16], u1[16], u2[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const unsigned short x0 =
                            *reinterpret_cast<const unsigned short *>(cp + (jb + j) * 128 + ((dc ^ (j & 7)) << 4));
                        const unsigned short x1 =
                            *reinterpret_cast<const unsigned short *>(cp + (jb + j + 1) * 128 + ((dc ^ ((j + 1) & 7)) << 4));
                        float y0 = __uint_as_float(static_cast<unsigned>(x0) << 16) * cw[jb + j];
                        float y1 = __uint_as_float(static_cast<unsigned>(x1) << 16) * cw[jb + j + 1];
                        const unsigned p0 = pack(y0, y1);
                        y0 -= lo_of(p0), y1 -= hi_of(p0);
                        const unsigned p1 = pack(y0, y1);
                        y0 -= lo_of(p1), y1 -= hi_of(p1);
                        u0[j / 2] = p0, u1[j / 2] = p1, u2[j / 2] = pack(y0, y1);
                    }
                    tmem_st16(tl + Y::T_V + jb / 2, u0);
                    tmem_st16(tl + Y::T_V + 64 + jb / 2, u1);
                    tmem_st16(tl + Y::T_V + 128 + jb / 2, u2);
                }
                tmem_st_wait();
                fence_before();
                __syncwarp();
                if (lane == 0) arrive(smem_u32(&bars->v));
                const float gn = rp[128 - n];
                if (!mbar_wait(smem_u32(&bars->ds), ph, err)) break;
                fence_after();
#pragma unroll
                for (int k = 0; k < KH; k += 32) {
                    float v[32];
                    tmem_ld32(t_ds + k, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) S[k + i] = fmaf(gn, S[k + i], w.update * v[i]);
                }
                fence_before();
                __syncwarp();
                if (lane == 0) arrive(smem_u32(&bars->ds_read));
                if (!STATE_ONLY) publish();
            }
            // the last state: segment's own (pass 1) or the sequence's
            const int last = L > 0 ? (L - 1) / w.seg : 0;
            float *p = nullptr;
            int si = w.dv;
            if (STATE_ONLY) {
                p = w.seg_state + (static_cast<long long>(bh) * w.n_seg + sg) * w.dk * w.dv + c0 + d;
            } else if (w.s_out != nullptr && sg == last) {
                p = w.s_out + static_cast<long long>(bh) * w.dk * w.dv + static_cast<long long>(c0 + d) * w.s_j;
                si = w.s_i;
            }
            if (p != nullptr && d < ncol) {
                const bool bad = *err != 0;
#pragma unroll
                for (int k = 0; k < KH; ++k)
                    if (half * KH + k < w.dk)
                        p[static_cast<long long>(half * KH + k) * si] = bad ? __int_as_float(0x7fc00000) : S[k];
            }
        }
    } else if (warp == 12) {
        // ---- the products
        if (lane == 0) {
            constexpr unsigned id_scores = make_idesc(1u, 128, kC), id_inter = make_idesc(1u, 128, DV);
            constexpr unsigned id_out = make_idesc(1u, 128, DV) | kNMajorB, id_ds = make_idesc(1u, 128, 64) | kNMajorB;
            bool ok = true;
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1;
                const unsigned ph = c & 1;
                const unsigned ta = sm + st * Y::STAGE + Y::A, tb = sm + st * Y::STAGE + Y::B, tc_ = sm + st * Y::STAGE + Y::C;
                if (!(ok = mbar_wait(smem_u32(&bars->full[st]), (c >> 1) & 1, err))) break;
                if (!STATE_ONLY) {
                    if (c > 0 && !(ok = mbar_wait(smem_u32(&bars->ds_read), ph ^ 1u, err))) break;
                    fence_after();
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k) {
                        const unsigned off = (k >> 2) * kPanel + (k & 3) * 32;
                        mma_ss(tm + Y::T_P, sw128_desc(ta + off), sw128_desc(tb + off), id_scores, k > 0);
                    }
                    commit(smem_u32(&bars->scores));
                    if (!(ok = mbar_wait(smem_u32(&bars->ss), ph, err))) break;
                    if (c > 0 && !(ok = mbar_wait(smem_u32(&bars->out_read), ph ^ 1u, err))) break;
                    fence_after();
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k)
                        mma_ss(tm + Y::T_O, sw128_desc(ta + (k >> 2) * kPanel + (k & 3) * 32),
                               sw128_desc(sm + Y::SS + (k >> 2) * (DV * 128) + (k & 3) * 32), id_inter, k > 0);
                    commit(smem_u32(&bars->inter));
                    if (!(ok = mbar_wait(smem_u32(&bars->p), ph, err))) break;
                    fence_after();
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k)
                        mma_ts(tm + Y::T_O, tm + Y::T_P + k * 8, nmajor_desc(tc_ + k * 2048), id_out, true);
                    commit(smem_u32(&bars->out));
                }
                if (!(ok = mbar_wait(smem_u32(&bars->v), ph, err))) break;
                fence_after();
#pragma unroll 1
                for (int term = 2; term >= 0; --term)  // smallest first
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k) {
                        const unsigned a = tm + Y::T_V + term * 64 + k * 8;
                        mma_ts(tm + Y::T_D0, a, nmajor_desc(tb + k * 2048), id_ds, term < 2 || k > 0);
                        if (DK == 128)
                            mma_ts(tm + Y::T_D1, a, nmajor_desc(tb + kPanel + k * 2048), id_ds, term < 2 || k > 0);
                    }
                commit(smem_u32(&bars->ds));
                commit(smem_u32(&bars->empty[st]));
            }
            // everything issued has finished before TMEM is given back
            commit(smem_u32(&bars->drain));
            mbar_drain(smem_u32(&bars->drain), 0);
        }
        __syncwarp();
    } else {
        // ---- copies
        const int lt = tid - 13 * 32;
        const __nv_bfloat16 *pa =
            static_cast<const __nv_bfloat16 *>(w.a.p) + b * w.a.sb + (h / w.a.group) * w.a.sh;
        const __nv_bfloat16 *pb =
            static_cast<const __nv_bfloat16 *>(w.b.p) + b * w.b.sb + (h / w.b.group) * w.b.sh;
        const __nv_bfloat16 *pc =
            static_cast<const __nv_bfloat16 *>(w.c.p) + b * w.c.sb + (h / w.c.group) * w.c.sh + c0;
        auto vec = [](const __nv_bfloat16 *p, long long st) {
            return reinterpret_cast<uintptr_t>(p) % 16 == 0 && st % 8 == 0;
        };
        const bool va = vec(pa, w.a.st), vb = vec(pb, w.b.st), vc = vec(pc, w.c.st);
        const int dir = w.reverse ? -1 : 1;
        for (int c = 0; c <= chunks; ++c) {
            if (c < chunks) {
                const int st = c & 1;
                if (c >= 2 && !mbar_wait(smem_u32(&bars->empty[st]), ((c >> 1) & 1) ^ 1u, err)) break;
                const int r0 = lo + c * kC, n = min(kC, hi - r0);
                const long long t0 = w.reverse ? L - 1 - r0 : r0;
                const unsigned base = sm + st * Y::STAGE;
                if (!STATE_ONLY) copy_tile<DK / 64>(base + Y::A, pa, w.a.st, t0, dir, n, w.dk, va, lt);
                copy_tile<DK / 64>(base + Y::B, pb, w.b.st, t0, dir, n, w.dk, vb, lt);
                copy_tile<DV / 64>(base + Y::C, pc, w.c.st, t0, dir, n, ncol, vc, lt);
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
            if (c > 0) {  // the chunk before has arrived
                if (c < chunks) asm volatile("cp.async.wait_group 1;" ::: "memory");
                else asm volatile("cp.async.wait_group 0;" ::: "memory");
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) arrive(smem_u32(&bars->full[(c - 1) & 1]));
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }

    fence_before();
    __syncthreads();
    if (warp == 12) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512));
    }
    if (!STATE_ONLY) {
        TO *po = static_cast<TO *>(w.out) + (static_cast<long long>(b) * w.T * w.H + h) * w.dv + c0;
        const long long ost = static_cast<long long>(w.H) * w.dv;
        if (*err)  // a wait ran out: nothing of this segment is to be trusted
            for (long long i = tid; i < static_cast<long long>(hi - lo) * ncol; i += kThreads) {
                const long long r = lo + i / ncol, t = w.reverse ? L - 1 - r : r;
                po[t * ost + i % ncol] = static_cast<TO>(__int_as_float(0x7fc00000));
            }
        // outputs behind the sequence's length are zero
        const long long t_lo = r_lo > L ? r_lo : L, t_hi = r_lo + w.seg < w.T ? r_lo + w.seg : w.T;
        for (long long i = tid; i < (t_hi - t_lo) * ncol; i += kThreads)
            po[(t_lo + i / ncol) * ost + i % ncol] = static_cast<TO>(0.f);
    }
}

template <typename TO, int DK, int DV, bool STATE_ONLY>
cudaError_t launch(const LaSweep &w, cudaStream_t s) {
    auto k = la_tc_kernel<TO, DK, DV, STATE_ONLY>;
    constexpr int smem = Lay<DK, DV>::BYTES > 120 * 1024 ? Lay<DK, DV>::BYTES : 120 * 1024;  // one CTA per SM (TMEM)
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // the last segment's own state is not needed
    const dim3 grid(static_cast<unsigned>(w.B) * w.H * ((w.dv + DV - 1) / DV), STATE_ONLY ? w.n_seg - 1 : w.n_seg);
    k<<<grid, kThreads, smem, s>>>(w);
    return cudaGetLastError();
}

template <typename TO, int DK, int DV>
cudaError_t sweep(const LaSweep &w, cudaStream_t s) {
    cudaError_t e;
    if (w.n_seg > 1) {
        if ((e = launch<TO, DK, DV, true>(w, s)) != cudaSuccess) return e;
        if ((e = launch_la_join(w, s)) != cudaSuccess) return e;
    }
    return launch<TO, DK, DV, false>(w, s);
}

template <typename TO>
cudaError_t by_width(const LaSweep &w, cudaStream_t s) {
    if (w.dk <= 64) return w.dv <= 64 ? sweep<TO, 64, 64>(w, s) : sweep<TO, 64, 128>(w, s);
    return w.dv <= 64 ? sweep<TO, 128, 64>(w, s) : sweep<TO, 128, 128>(w, s);
}

}  // namespace

cudaError_t launch_la_tc(const LaSweep &w, cudaStream_t s) {
    return w.out_f32 ? by_width<float>(w, s) : by_width<__nv_bfloat16>(w, s);
}

}  // namespace pararnn
