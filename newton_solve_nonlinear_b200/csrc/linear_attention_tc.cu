// linear_attention_tc.cu -- the sweep of linear_attention.cuh for bf16 operands on the 5th-generation tensor
// cores (tcgen05, sm_100a).
//
// One CTA carries one head's state through one segment of time, 128 rows at a time:
//   scores = a b^T                      [128 x 128]  operands in shared memory
//   out    = g^(i+e) (a S)              [128 x DV]   S as a bf16 copy in shared memory
//   out   += (scores * g^(i-j)) c       [128 x DV]   weighted scores rounded to bf16 in TMEM as the A operand
//   dS^T   = (g^(n-e-j) c)^T b          [DV x DK]    weighted c in TMEM as the A operand
//   S      = g^n S + dS                 in registers, fp32
// A bf16 product is exact in fp32, so the only roundings below fp32 are those of the weighted scores and of S's
// copy, each at most 2^-8 relative as the output's own.  The weighted c is split into three bf16 terms (24 bits), so the
// state's products are exact to fp32; they are summed smallest term first.
//
// Tiles are of 128 consecutive tokens from a multiple of 128 on, in the order of the tokens.  A reversed sweep
// takes them from the last one down and mirrors the weights (logical row = n - 1 - tile row), so tiles come and go
// by TMA either way, and only the tile with the sequence's end is not full.
//
// Warps: 0-7 output (lane quarter = rows, two halves of the columns: weigh the scores, scale, stage for the TMA
// store), 8-15 state (lane quarter = columns of c; two halves of the rows to be split and of b's width), 16
// issues the products, 17 moves the tiles (two stages).  Every wait is bounded; a wait that runs out marks this
// CTA's results NaN.
//
// Measured on 8 x 8192 tokens, 16 heads of 128: 229 us alone on the GPU, 0.72 of a copy of its bytes; the tensor pipe is
// busy 44 % of the time.  It is bound by the chain of a chunk, about 6300 cycles with 128 columns: split of the weighted c
// (2800, with the scores' weighing beside it), products (1900), state update and its copy (700), which the next chunk's
// products wait for.  Two chunks in flight would hide it, but at this width one fills 227 KB of shared memory and all 512
// columns of TMEM.  128 tokens are one row of products for each TMEM lane.  Sixteen state warps with a quarter of the
// work each gave 236 us: 72 registers a thread are too few for the output warps.  The 128-wide kernels use local memory
// beside their registers, 96 bytes of stores a thread (268 in the state-only pass).
#include <cuda_bf16.h>

#include "linear_attention.cuh"
#include "tc_utils.cuh"

namespace pararnn {
namespace {
using namespace tc;

constexpr int kC = 128;       // rows per chunk
// Five warpgroups of 96 registers a thread at launch, 61440 in all; the state's two take 128 of them each thread
// (S is 64), the outputs' two keep 88 and the last one 48: 256 * 128 + 256 * 88 + 128 * 48 = 61440.
constexpr int kThreads = 20 * 32;
constexpr int kRegsState = 128, kRegsOut = 88, kRegsMove = 48;
static_assert(256 * kRegsState + 256 * kRegsOut + 128 * kRegsMove <= kThreads * 96, "register split");
constexpr int kPanel = kC * 128;  // bytes of a [128 rows][64 bf16] panel

template <int DK, int DV>
struct Lay {
    static constexpr int A = 0, B = A + DK / 64 * kPanel, C = B + DK / 64 * kPanel, END = C + DV / 64 * kPanel;
    // a is free once both of its products are done: the outputs are staged there, if it is wide enough
    static constexpr int OUT = DV <= DK ? A : END, STAGE = DV <= DK ? END : END + DV / 64 * kPanel;
    static constexpr int SS = 2 * STAGE;                 // bf16 S: [DV rows][DK], K-major panels
    static constexpr int TAB = SS + DK / 64 * DV * 128;  // floats: score weights 160, row weights 2 x 160
    static constexpr int BARS = TAB + (160 + 320) * 4;
    static constexpr int BYTES = BARS + 136 + 1008;  // + alignment, from 16 bytes up
    // TMEM columns: scores, each half of which becomes the weighted scores of its 64 columns (32-bit columns 0-31 and
    // 64-95); out; dS; the weighted c's terms, smallest first, 64 columns each.  With DK = DV = 128 there is no room for
    // the third: it takes the columns that the weighted scores leave free (32-63 and 96-127), once the scores have been
    // read, and the next scores wait for its use.  Pass 1 has neither scores nor outputs: dS and two sets of terms, so
    // that the next chunk is split while this one's products run.
    static constexpr bool ROOM = DK + DV <= 192;
    static constexpr int T_S = 0, T_O = 128, T_D = 128 + DV, T_V = T_D + DK;
    static constexpr int T_D1 = 0, T_V1 = 128;
    static constexpr int STATE_WARPS = 8;
    // lane of column d of c, as a row of dS: with 64 columns, 16 in each warp's quarter, so that all warps have some
    static constexpr int ROWS = DV / 4;
    static_assert(BYTES <= 227 * 1024, "shared memory");
};

struct Bars {
    unsigned long long full[2], empty[2], staged[2], scores, inter, p, scaled, v, ss, out, ds, out_read, clean;
    unsigned tmem;
    int err;
};
static_assert(sizeof(Bars) <= 136, "barriers");

// A barrier's next phase completes only after everyone who waits for this one has seen it (the parity would be
// ambiguous otherwise): the chains scores -> p -> scaled -> out -> scores and v -> ds -> v order all but the mover,
// whose barriers are one per stage, and a stage is filled again only by the mover itself.

// One sweep's arguments: its sizes and pointers, and the tensor maps of its tiles.
struct TcSweep {
    LaSweep w;
    CUtensorMap a, b, c, out;
};
struct TcBatch {
    TcSweep s[3];
};

__device__ __forceinline__ void arrive(unsigned bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void commit(unsigned bar, unsigned on) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(on));
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

template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ bool elect_one() {
    unsigned r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0u;
}

// The warp runs these together and one lane (`on`) issues: without a branch the operands stay in uniform registers.
__device__ __forceinline__ void mma_ss(unsigned d, unsigned long long a, unsigned long long b, unsigned idesc, bool acc,
                                       unsigned on) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(on));
}
__device__ __forceinline__ void mma_ts(unsigned d, unsigned a, unsigned long long b, unsigned idesc, bool acc,
                                       unsigned on) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(on));
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
// (a, b) = (a, b) * (x, y), and = (a, b) * g + (x, y): two fp32 lanes at a time
__device__ __forceinline__ void mul2(float &a, float &b, float x, float y) {
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(x), "f"(y));
}
__device__ __forceinline__ void fma2(float &a, float &b, float g, float x, float y) {
    asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tmov.b64 r, {%3, %4};\n\t"
        "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(g), "f"(x), "f"(y));
}
// (a, b) -= (x, y), exactly as two subtractions
__device__ __forceinline__ void sub2(float &a, float &b, float x, float y) {
    fma2(x, y, -1.f, a, b);
    a = x, b = y;
}

__device__ __forceinline__ float lo_of(unsigned u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_of(unsigned u) { return __uint_as_float(u & 0xffff0000u); }

// The weighted c's 16 x (2 x 8) pieces: .16x128b holds row lane / 4 (+ 8 in odd registers), 32-bit column lane % 4 of
// each group of four, which is the fragment that a transposed ldmatrix of [tokens][columns] delivers.
__device__ __forceinline__ void tmem_st_frag(unsigned addr, const unsigned (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}
__device__ __forceinline__ void ldmatrix4t(unsigned addr, unsigned &a, unsigned &b, unsigned &c, unsigned &d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void tma_load_4d(unsigned dst, const CUtensorMap *map, int x, int t, int h, int b, unsigned bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<unsigned long long>(map)), "r"(x), "r"(t), "r"(h), "r"(b), "r"(bar)
        : "memory");
}
// Brings a tile into L2 ahead of its load.
__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap *map, int x, int t, int h, int b) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                     reinterpret_cast<unsigned long long>(map)),
                 "r"(x), "r"(t), "r"(h), "r"(b)
                 : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap *map, int x, int t, int h, int b, unsigned src) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                     reinterpret_cast<unsigned long long>(map)),
                 "r"(x), "r"(t), "r"(h), "r"(b), "r"(src)
                 : "memory");
}

// 32 columns of one output row of a padded width (a multiple of 8).
__device__ __forceinline__ void store32(float *p, const float (&v)[32], int room) {
#pragma unroll
    for (int i = 0; i < 32; i += 4)
        if (i < room) *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}

template <int DK, int DV, bool STATE_ONLY>
__global__ void __launch_bounds__(kThreads, 1) la_tc_kernel(const __grid_constant__ TcBatch batch) {
    using Y = Lay<DK, DV>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                            ~static_cast<uintptr_t>(1023));
    const TcSweep &sweep = batch.s[blockIdx.z];
    const LaSweep &w = sweep.w;
    const unsigned sm = smem_u32(smem);
    // weight of the score (row x, column y), intra g^|x - y| or 0, at sw[y - x]: of y - x in -127 .. 32 forward, in
    // -32 .. 127 reversed, as far as any block needs it
    float *sw = reinterpret_cast<float *>(smem + Y::TAB);
    // update g^(n - e - j) of tile row x, for a full tile and for the last one: [2][8][20], row x = 64 h + 8 g + 2 l + i
    // at [4 h + l][2 g + i], the order in which a lane of the state warps wants them (rows 20 apart: no bank conflicts); in
    // the first gap, at 16, what rounding leaves of g^n for a full tile
    float *cw = sw + 160;
    Bars *bars = reinterpret_cast<Bars *>(smem + Y::BARS);
    volatile int *err = &bars->err;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int bh = blockIdx.x, b = bh / w.H, h = bh % w.H, sg = blockIdx.y;
    int L = w.T;
    if (w.lengths != nullptr) L = min(max(w.lengths[b], 0), w.T);
    // tokens [lo, hi) of this segment; the tile with hi has n_part rows
    const long long t_lo = static_cast<long long>(sg) * w.seg;
    const int lo = t_lo < L ? static_cast<int>(t_lo) : L;
    const int hi = t_lo + w.seg < L ? static_cast<int>(t_lo + w.seg) : L;
    const int chunks = (hi - lo + kC - 1) / kC;
    const int n_part = hi - lo - (chunks - 1) * kC;
    const bool rev = w.reverse != 0;
    const int e = w.e;
    const int part_chunk = rev ? 0 : chunks - 1;
    const bool unclean = chunks > 0 && n_part < kC;  // rows to be cleared: behind the sequence's end
    const float ld = safe_log_decay(w.log_decay[h]);
    auto power = [&](int n) { return decay_pow(ld, n); };
    // first token of chunk c's tile
    auto first_token = [&](int c) { return lo + (rev ? chunks - 1 - c : c) * kC; };

    if (STATE_ONLY && sg == (rev ? 0 : w.n_seg - 1)) return;
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&bars->full[s]), STATE_ONLY ? 1 : 2);
            mbar_init(smem_u32(&bars->empty[s]), 1);
            mbar_init(smem_u32(&bars->staged[s]), 8);
        }
        mbar_init(smem_u32(&bars->scores), 1);
        mbar_init(smem_u32(&bars->inter), 1);
        mbar_init(smem_u32(&bars->out), 1);
        mbar_init(smem_u32(&bars->ds), 1);
        mbar_init(smem_u32(&bars->p), 8);
        mbar_init(smem_u32(&bars->clean), Y::STATE_WARPS);
        mbar_init(smem_u32(&bars->scaled), 8);
        mbar_init(smem_u32(&bars->out_read), 8);
        mbar_init(smem_u32(&bars->v), Y::STATE_WARPS);
        mbar_init(smem_u32(&bars->ss), Y::STATE_WARPS);
        bars->err = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 16) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid < 160) {
        const int x = rev ? tid - 32 : 127 - tid;  // row distance, counted towards the past
        sw[tid] = x >= 0 ? power(x) * w.intra : 0.f;
    } else if (tid < 160 + 256) {
        const int x = (tid - 160) & 127, n = tid - 160 < 128 ? kC : n_part, j = rev ? n - 1 - x : x;
        cw[(tid - 160 < 128 ? 0 : 160) + ((x >> 6) * 4 + ((x & 7) >> 1)) * 20 + ((x & 63) >> 3) * 2 + (x & 1)] =
            x < n ? power(n - e - j) * w.update : 0.f;
    } else if (tid == 160 + 256) {
        cw[16] = decay_rest(ld, kC);
    }
    fence_before();
    __syncthreads();
    fence_after();
    const unsigned tm = bars->tmem;

    if (warp < 8) {
        // ---- outputs: thread = tile row, half = half of the columns
        regs_down<kRegsOut>();
        if (!STATE_ONLY) {
            const int quarter = warp & 3, half = warp >> 2, row = quarter * 32 + lane;
            const unsigned tl = tm + (static_cast<unsigned>(quarter * 32) << 16);
            auto row_factor = [&](int n) { return power((rev ? n - 1 - row : row) + e) * w.inter; };
            const float f_full = row_factor(kC), f_part = row < n_part ? row_factor(n_part) : 0.f;
            // fp32 outputs (partial gradients): dense rows of w.out_w columns
            const long long ost = static_cast<long long>(w.H) * w.out_w;
            float *const pf = w.out_f32 ? static_cast<float *>(w.out) +
                                              (static_cast<long long>(b) * w.T * w.H + h) * w.out_w + row * ost
                                        : nullptr;
            for (int c = 0; c < chunks; ++c) {
                const unsigned ph = c & 1;
                const bool full = c != part_chunk;
                const float f = full ? f_full : f_part;
                if (!mbar_wait(smem_u32(&bars->scores), ph, err)) break;
                fence_after();
#pragma unroll 1
                for (int jb = half * 2; jb < half * 2 + 2; ++jb) {
                    unsigned u[16] = {};
                    if (rev ? jb >= quarter : jb <= quarter) {  // else all of the block is masked
                        float v[32];
                        tmem_ld32(tl + Y::T_S + jb * 32, v);
                        const float *s = sw + (rev ? 32 : 127) + jb * 32 - row;
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            mul2(v[j], v[j + 1], s[j], s[j + 1]);
                            u[j / 2] = pack(v[j], v[j + 1]);
                        }
                    }
                    // in the place of scores that this warp has read
                    tmem_st16(tl + Y::T_S + half * 64 + (jb & 1) * 16, u);
                }
                if (!Y::ROOM) {  // the state warps may write where scores were
                    tmem_st_wait();
                    fence_before();
                    __syncwarp();
                    if (lane == 0) arrive(smem_u32(&bars->p));
                }
                if (!mbar_wait(smem_u32(&bars->inter), ph, err)) break;
                fence_after();
#pragma unroll 1
                for (int cb = half * (DV / 2); cb < (half + 1) * (DV / 2); cb += 32) {
                    float v[32];
                    tmem_ld32(tl + Y::T_O + cb, v);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) mul2(v[j], v[j + 1], f, f);
                    tmem_st32(tl + Y::T_O + cb, v);
                }
                tmem_st_wait();
                fence_before();
                __syncwarp();
                if (lane == 0) arrive(smem_u32(&bars->scaled));
                if (!mbar_wait(smem_u32(&bars->out), ph, err)) break;
                fence_after();
                const bool live = full || row < n_part;
#pragma unroll 1
                for (int cb = half * (DV / 2); cb < (half + 1) * (DV / 2); cb += 32) {
                    float v[32];
                    tmem_ld32(tl + Y::T_O + cb, v);
                    if (cb == (half + 1) * (DV / 2) - 32) {
                        fence_before();
                        __syncwarp();
                        if (lane == 0) arrive(smem_u32(&bars->out_read));
                    }
                    if (pf != nullptr) {
                        if (live) store32(pf + first_token(c) * ost + cb, v, w.out_w - cb);
                    } else {
                        if (!live) {
#pragma unroll
                            for (int q = 0; q < 32; ++q) v[q] = 0.f;
                        }
                        const unsigned at = sm + (c & 1) * Y::STAGE + Y::OUT + (cb >> 6) * kPanel + row * 128;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const unsigned d = at + (((((cb & 32) >> 3) + q) ^ (row & 7)) << 4);
                            unsigned u[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) u[k] = pack(v[8 * q + 2 * k], v[8 * q + 2 * k + 1]);
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(d), "r"(u[0]), "r"(u[1]),
                                         "r"(u[2]), "r"(u[3])
                                         : "memory");
                        }
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) arrive(smem_u32(&bars->staged[c & 1]));
            }
        }
    } else if (warp < 16) {
        // ---- state: TMEM lane = column of c; half = half of b's width and of the chunk's rows
        regs_up<kRegsState>();
        const int quarter = warp & 3, half = (warp - 8) >> 2;
        {
            constexpr int KH = DK / 2;
            constexpr bool HOLES = !STATE_ONLY && !Y::ROOM;  // the largest term stands between the weighted scores
            const int d = quarter * Y::ROWS + (lane & (Y::ROWS - 1));  // with 64 columns, lanes 16-31 have none
            const bool mine = lane < Y::ROWS;
            const unsigned tl = tm + (static_cast<unsigned>(quarter * 32) << 16);
            const unsigned t_ds = tl + (STATE_ONLY ? Y::T_D1 : Y::T_D) + half * KH;
            float S[KH];
            {
                const bool have = mine && d < w.dv && (w.n_seg > 1 ? !STATE_ONLY : w.s_in != nullptr);
                const float *p = w.n_seg > 1
                                     ? w.seg_state + (static_cast<long long>(bh) * w.n_seg + sg) * w.dk * w.dv + d
                                     : w.s_in + static_cast<long long>(bh) * w.dk * w.dv +
                                           static_cast<long long>(d) * w.s_j;
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
                    if (!mine) break;
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
            // ldmatrix: lane l names row l % 8 of matrix l / 8; matrices are (8 tokens) x (8 columns of c), columns
            // first, then tokens
            const int m_row = half * 64 + ((lane >> 4) << 3) + (lane & 7);
            const float g_full = power(kC), g_part = power(n_part);
            // S = g^n S + dS of chunk c.  What rounding leaves of g^n is handed from full tile to full tile and taken when it
            // makes a step of the weight, so that the weights' product is off by one rounding and not by one a chunk
            float owed = 0.f;
            auto absorb = [&](int c) {
                float gn = g_part;
                if (c != part_chunk) {
                    owed += cw[16];
                    gn = g_full + owed;
                    owed -= gn - g_full;
                }
                if (!mbar_wait(smem_u32(&bars->ds), c & 1, err)) return false;
                fence_after();
#pragma unroll
                for (int k = 0; k < KH; k += 32) {
                    float v[32];
                    tmem_ld32(t_ds + k, v);
#pragma unroll
                    for (int q = 0; q < 32; q += 2) fma2(S[k + q], S[k + q + 1], gn, v[q], v[q + 1]);
                }
                fence_before();
                return true;
            };
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1;
                const unsigned ph = c & 1;
                const bool part = c == part_chunk;
                const unsigned tile_b = sm + st * Y::STAGE + Y::B, tile_c = sm + st * Y::STAGE + Y::C;
                if (!mbar_wait(smem_u32(&bars->full[st]), (c >> 1) & 1, err)) break;
                const int col0 = quarter * Y::ROWS;  // this warp's columns of c
                const unsigned panel_c = tile_c + (col0 >> 6) * kPanel;
                if (part && unclean) {  // tokens behind the sequence's end: this warp's share of c, and of b
                    constexpr int CH = Y::ROWS / 8;
                    for (int x = max(n_part, half * 64) + lane / CH; x < half * 64 + 64; x += 32 / CH) {
                        const int ch = ((col0 & 63) >> 3) + lane % CH;
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(panel_c + x * 128 +
                                                                                      ((ch ^ (x & 7)) << 4)),
                                     "r"(0)
                                     : "memory");
                    }
                    const int me = half * 4 + quarter;
                    for (int x = n_part + me; x < kC; x += Y::STATE_WARPS)
                        if (lane < DK / 8)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             tile_b + (lane >> 3) * kPanel + x * 128 + (((lane & 7) ^ (x & 7)) << 4)),
                                         "r"(0)
                                         : "memory");
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) arrive(smem_u32(&bars->clean));
                }
                const float *cwt = cw + (part ? 160 : 0) + (half * 4 + (lane & 3)) * 20;
                const unsigned ta = tl + (STATE_ONLY ? Y::T_V1 + (c & 1) * 192 : Y::T_V) + half * 32;
                // 16 columns of c (sub), 64 tokens; registers k, k + 1: the same 8 tokens, columns lane / 4 and + 8
                auto load_c = [&](int sub, unsigned (&u)[16]) {
                    const int ch = ((col0 & 63) >> 3) + sub * 2 + ((lane >> 3) & 1);
                    const unsigned at = panel_c + m_row * 128 + ((ch ^ (lane & 7)) << 4);
#pragma unroll
                    for (int tb = 0; tb < 4; ++tb)
                        ldmatrix4t(at + tb * 2048, u[4 * tb], u[4 * tb + 1], u[4 * tb + 2], u[4 * tb + 3]);
                };
                bool seen = true;
#pragma unroll 1
                for (int sub = 0; sub < Y::ROWS / 16; ++sub) {
                    unsigned u0[16], u1[16], u2[16];
                    load_c(sub, u1);
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const float4 f4 = *reinterpret_cast<const float4 *>(cwt + (q >> 2) * 4);
                        const float f0 = q & 2 ? f4.z : f4.x, f1 = q & 2 ? f4.w : f4.y;
                        float y0 = lo_of(u1[q]), y1 = hi_of(u1[q]);
                        mul2(y0, y1, f0, f1);
                        u0[q] = pack(y0, y1);
                        sub2(y0, y1, lo_of(u0[q]), hi_of(u0[q]));
                        u1[q] = pack(y0, y1);
                        sub2(y0, y1, lo_of(u1[q]), hi_of(u1[q]));
                        u2[q] = pack(y0, y1);
                    }
                    const unsigned tsub = ta + (static_cast<unsigned>(sub * 16) << 16);
                    tmem_st_frag(tsub, u2);
                    tmem_st_frag(tsub + 64, u1);
                    if (HOLES) {
                        if (sub == 0 && !(seen = mbar_wait(smem_u32(&bars->p), ph, err))) break;
                        fence_after();
                        tmem_st_frag(tl + (static_cast<unsigned>(sub * 16) << 16) + Y::T_S + half * 64 + 32, u0);
                    } else {
                        tmem_st_frag(tsub + 128, u0);
                    }
                }
                if (!seen || (STATE_ONLY && c > 0 && !absorb(c - 1))) break;
                tmem_st_wait();
                fence_before();
                __syncwarp();
                if (lane == 0) arrive(smem_u32(&bars->v));
                if (!STATE_ONLY) {
                    if (!absorb(c)) break;
                    publish();
                }
            }
            if (STATE_ONLY && chunks > 0) absorb(chunks - 1);
            // the last state: the segment's own (pass 1) or the sequence's
            const int last_seg = L > 0 && !rev ? (L - 1) / w.seg : 0;
            float *p = nullptr;
            int si = w.dv;
            if (STATE_ONLY) {
                p = w.seg_state + (static_cast<long long>(bh) * w.n_seg + sg) * w.dk * w.dv + d;
            } else if (w.s_out != nullptr && sg == last_seg) {
                p = w.s_out + static_cast<long long>(bh) * w.dk * w.dv + static_cast<long long>(d) * w.s_j;
                si = w.s_i;
            }
            if (p != nullptr && mine && d < w.dv) {
                const bool bad = *err != 0;
#pragma unroll
                for (int k = 0; k < KH; ++k)
                    if (half * KH + k < w.dk)
                        p[static_cast<long long>(half * KH + k) * si] = bad ? __int_as_float(0x7fc00000) : S[k];
            }
        }
    } else {
    regs_down<kRegsMove>();
    if (warp == 16) {
        // ---- the products
        constexpr unsigned id_scores = make_idesc(1u, 128, kC), id_inter = make_idesc(1u, 128, DV);
        constexpr unsigned id_out = make_idesc(1u, 128, DV) | kNMajorB, id_ds = make_idesc(1u, 128, DK) | kNMajorB;
        const unsigned on = elect_one() ? 1u : 0u;
        const unsigned tu = __shfl_sync(0xffffffffu, tm, 0);
        constexpr bool HOLES = !STATE_ONLY && !Y::ROOM;
        int done = 0;  // chunks issued whole
        auto scores = [&](int c) {
            const unsigned ta = sm + (c & 1) * Y::STAGE + Y::A, tb = sm + (c & 1) * Y::STAGE + Y::B;
#pragma unroll 2
            for (int k = 0; k < DK / 16; ++k) {
                const unsigned off = (k >> 2) * kPanel + (k & 3) * 32;
                mma_ss(tu + Y::T_S, sw128_desc(ta + off), sw128_desc(tb + off), id_scores, k > 0, on);
            }
            commit(smem_u32(&bars->scores), on);
        };
        auto term = [&](int c, int place, bool first) {
            const unsigned tb = sm + (c & 1) * Y::STAGE + Y::B;
            const unsigned td = tu + (STATE_ONLY ? Y::T_D1 : Y::T_D);
            const unsigned tv = tu + (STATE_ONLY ? Y::T_V1 + (c & 1) * 192 : Y::T_V) + place * 64;
#pragma unroll 2
            for (int k = 0; k < kC / 16; ++k) {
                const unsigned ta = HOLES && place == 2 ? tu + Y::T_S + 32 + (k >> 2) * 64 + (k & 3) * 8 : tv + k * 8;
                mma_ts(td, ta, nmajor_desc(tb + k * 2048), id_ds, !first || k > 0, on);
            }
        };
        // scores of the tile whose rows the state warps clear wait for that
        if (chunks > 0 && mbar_wait(smem_u32(&bars->full[0]), 0, err) &&
            !(part_chunk == 0 && unclean && !mbar_wait(smem_u32(&bars->clean), 0, err))) {
            fence_after();
            if (!STATE_ONLY) scores(0);
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1;
                const unsigned ph = c & 1;
                const unsigned ta = sm + st * Y::STAGE + Y::A, tc_ = sm + st * Y::STAGE + Y::C;
                if (!STATE_ONLY) {
                    if (!mbar_wait(smem_u32(&bars->ss), ph, err)) break;
                    if (c > 0 && !mbar_wait(smem_u32(&bars->out_read), ph ^ 1u, err)) break;
                    fence_after();
#pragma unroll 2
                    for (int k = 0; k < DK / 16; ++k)
                        mma_ss(tu + Y::T_O, sw128_desc(ta + (k >> 2) * kPanel + (k & 3) * 32),
                               sw128_desc(sm + Y::SS + (k >> 2) * (DV * 128) + (k & 3) * 32), id_inter, k > 0, on);
                    commit(smem_u32(&bars->inter), on);
                }
                // dS, the smallest term first; dS's place is free: v comes after the state warps have read it
                auto state_products = [&]() {
                    if (!mbar_wait(smem_u32(&bars->v), ph, err)) return false;
                    fence_after();
                    term(c, 0, true);
                    term(c, 1, false);
                    term(c, 2, false);
                    commit(smem_u32(&bars->ds), on);
                    return true;
                };
                // which comes first is which operand is ready first
                if (!HOLES && !state_products()) break;
                if (!STATE_ONLY) {
                    if (!mbar_wait(smem_u32(&bars->scaled), ph, err)) break;
                    fence_after();
#pragma unroll 2
                    for (int k = 0; k < kC / 16; ++k)
                        mma_ts(tu + Y::T_O, tu + Y::T_S + (k >> 2) * 64 + (k & 3) * 8, nmajor_desc(tc_ + k * 2048), id_out,
                               true, on);
                    commit(smem_u32(&bars->out), on);
                }
                if (HOLES && !state_products()) break;
                commit(smem_u32(&bars->empty[st]), on);
                done = c + 1;
                if (c + 1 < chunks) {
                    if (!mbar_wait(smem_u32(&bars->full[st ^ 1]), ((c + 1) >> 1) & 1, err)) break;
                    if (!STATE_ONLY) {  // the next scores, as soon as the weighted ones have been used
                        if (!mbar_wait(smem_u32(&bars->out), ph, err)) break;
                        if (HOLES && !mbar_wait(smem_u32(&bars->ds), ph, err)) break;
                        if (c + 1 == part_chunk && unclean && !mbar_wait(smem_u32(&bars->clean), 0, err)) break;
                        fence_after();
                        scores(c + 1);
                    }
                }
            }
        }
        // everything issued has finished before TMEM is given back: each chunk's last commit, or, where a wait ran
        // out in the middle of a chunk, a last one
        if (*err) {
            const int st = done & 1;
            commit(smem_u32(&bars->empty[st]), on);
            mbar_drain(smem_u32(&bars->empty[st]), (done >> 1) & 1);
        } else if (done > 0) {
            mbar_drain(smem_u32(&bars->empty[(done - 1) & 1]), ((done - 1) >> 1) & 1);
        }
    } else if (warp == 17) {
        // ---- tiles in, staged outputs out
        const int ha = h / w.a.group, hb = h / w.b.group, hc = h / w.c.group;
        const bool f32 = w.out_f32 != 0;
        // first b and c, then a, whose place the staged outputs may hold longer
        auto load = [&](int c, bool first) {
            const int st = c & 1, t0 = first_token(c);
            const unsigned base = sm + st * Y::STAGE, full = smem_u32(&bars->full[st]);
            if (elect_one()) {
                if (first) {
                    mbar_expect_tx(full, (DK / 64 + DV / 64) * kPanel);
#pragma unroll
                    for (int x = 0; x < DV / 64; ++x)
                        tma_load_4d(base + Y::C + x * kPanel, &sweep.c, x * 64, t0, hc, b, full);
#pragma unroll
                    for (int x = 0; x < DK / 64; ++x)
                        tma_load_4d(base + Y::B + x * kPanel, &sweep.b, x * 64, t0, hb, b, full);
                } else {
                    mbar_expect_tx(full, DK / 64 * kPanel);
#pragma unroll
                    for (int x = 0; x < DK / 64; ++x)
                        tma_load_4d(base + Y::A + x * kPanel, &sweep.a, x * 64, t0, ha, b, full);
                }
            }
            __syncwarp();
        };
        // With small tiles two stages hold too few bytes in flight for DRAM's latency: tiles go to L2 a chunk before
        // their load (131072 tokens, 8 heads of 64: 207 -> 193 us; with 128 columns it is no gain: 234 -> 244 us on
        // 8 x 8192 x 16 heads)
        constexpr int kAhead = DK + DV <= 128 ? 1 : 0;
        auto prefetch = [&](int c) {
            if (elect_one()) {
                const int t0 = first_token(c);
#pragma unroll
                for (int x = 0; x < DV / 64; ++x) tma_prefetch_4d(&sweep.c, x * 64, t0, hc, b);
#pragma unroll
                for (int x = 0; x < DK / 64; ++x) {
                    tma_prefetch_4d(&sweep.b, x * 64, t0, hb, b);
                    if (!STATE_ONLY) tma_prefetch_4d(&sweep.a, x * 64, t0, ha, b);
                }
            }
            __syncwarp();
        };
        for (int c = 2; c < min(chunks, 2 + kAhead); ++c) prefetch(c);
        int loaded = 0;  // chunks of which any tile was asked for
#pragma unroll 1
        for (int c = -2; c < chunks; ++c) {
            if (c + 2 < chunks) {
                if (c >= 0 && !mbar_wait(smem_u32(&bars->empty[c & 1]), (c >> 1) & 1, err)) break;
                load(c + 2, true);
                loaded = c + 3;
                if (kAhead > 0 && c >= 0 && c + 2 + kAhead < chunks) prefetch(c + 2 + kAhead);
            }
            if (STATE_ONLY) continue;
            if (c >= 0) {
                if (!mbar_wait(smem_u32(&bars->staged[c & 1]), (c >> 1) & 1, err)) break;
                if (!f32) {
                    if (elect_one()) {
#pragma unroll
                        for (int x = 0; x < DV / 64; ++x)
                            if (x * 64 < w.dv)
                                tma_store_4d(&sweep.out, x * 64, first_token(c), h, b,
                                             sm + (c & 1) * Y::STAGE + Y::OUT + x * kPanel);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        // the store has read its tile before the stage is filled again
                        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    }
                    __syncwarp();
                }
            }
            if (c + 2 < chunks) load(c + 2, false);
        }
        if (*err) {  // copies in flight land before the block ends
            for (int c = max(loaded - 2, 0); c < loaded; ++c) mbar_drain(smem_u32(&bars->full[c & 1]), (c >> 1) & 1);
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    }

    fence_before();
    __syncthreads();
    if (warp == 16) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512));
    }
    if (!STATE_ONLY) {
        const long long po = (static_cast<long long>(b) * w.T * w.H + h) * w.out_w;
        const long long ost = static_cast<long long>(w.H) * w.out_w;
        auto put = [&](long long at, float x) {
            if (w.out_f32) static_cast<float *>(w.out)[at] = x;
            else static_cast<__nv_bfloat16 *>(w.out)[at] = __float2bfloat16(x);
        };
        if (*err)  // a wait ran out: nothing of this segment is to be trusted
            for (long long i = tid; i < static_cast<long long>(hi - lo) * w.dv; i += kThreads)
                put(po + (lo + i / w.dv) * ost + i % w.dv, __int_as_float(0x7fc00000));
        // outputs behind the sequence's length are zero
        const long long z_lo = t_lo > L ? t_lo : L, z_hi = t_lo + w.seg < w.T ? t_lo + w.seg : w.T;
        for (long long i = tid; i < (z_hi - z_lo) * w.dv; i += kThreads) put(po + (z_lo + i / w.dv) * ost + i % w.dv, 0.f);
    }
}

// A [B, T, heads, width] operand in boxes of 128 tokens x 64 columns.
bool make_rows_map(CUtensorMap *m, const void *p, int B, int T, int heads, int width, long long sb, long long st,
                   long long sh) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const long long n[3] = {T, heads, B};
    const long long s[3] = {st, sh, sb};
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(width), 0, 0, 0}, strides[3];
    for (int i = 0; i < 3; ++i) {
        dims[i + 1] = static_cast<cuuint64_t>(n[i]);
        strides[i] = n[i] > 1 ? static_cast<cuuint64_t>(s[i]) * 2 : 256;  // an axis of one entry is never stepped
    }
    const cuuint32_t box[4] = {64, kC, 1, 1}, one[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool with_maps(const LaSweep &w, TcSweep *t) {
    t->w = w;
    auto in = [&](CUtensorMap *m, const LaRows &r, int width) {
        return make_rows_map(m, r.p, w.B, w.T, w.H / r.group, width, r.sb, r.st, r.sh);
    };
    const long long row = static_cast<long long>(w.H) * w.out_w;
    return in(&t->a, w.a, w.dk) && in(&t->b, w.b, w.dk) && in(&t->c, w.c, w.dv) &&
           (w.out_f32 || make_rows_map(&t->out, w.out, w.B, w.T, w.H, w.out_w, w.T * row, row, w.out_w));
}

template <int DK, int DV, bool STATE_ONLY>
cudaError_t launch(const TcBatch &t, int n, cudaStream_t s) {
    auto k = la_tc_kernel<DK, DV, STATE_ONLY>;
    constexpr int smem = Lay<DK, DV>::BYTES > 120 * 1024 ? Lay<DK, DV>::BYTES : 120 * 1024;  // one CTA per SM (TMEM)
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const LaSweep &w = t.s[0].w;
    // pass 1: the state of the segment that comes last is not needed (its blocks return at once)
    const dim3 grid(static_cast<unsigned>(w.B) * w.H, w.n_seg, n);
    k<<<grid, kThreads, smem, s>>>(t);
    return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t sweep(const TcBatch &t, int n, cudaStream_t s) {
    cudaError_t e;
    if (t.s[0].w.n_seg > 1) {
        if ((e = launch<DK, DV, true>(t, n, s)) != cudaSuccess) return e;
        for (int i = 0; i < n; ++i)
            if ((e = launch_la_join(t.s[i].w, s)) != cudaSuccess) return e;
    }
    return launch<DK, DV, false>(t, n, s);
}

cudaError_t by_width(const TcBatch &t, int n, cudaStream_t s) {
    const LaSweep &w = t.s[0].w;
    if (w.dk <= 64) return w.dv <= 64 ? sweep<64, 64>(t, n, s) : sweep<64, 128>(t, n, s);
    return w.dv <= 64 ? sweep<128, 64>(t, n, s) : sweep<128, 128>(t, n, s);
}

}  // namespace

cudaError_t launch_la_tc(const LaSweep *w, int n, cudaStream_t s) {
    TcBatch t{};
    for (int i = 0; i < n; ++i)
        if (!with_maps(w[i], &t.s[i])) return cudaErrorInvalidValue;
    return by_width(t, n, s);
}

bool la_tc_readable(const LaRows &r, int B, int T, int heads) {
    const long long n[3] = {T, heads, B}, s[3] = {r.st, r.sh, r.sb};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (s[i] == 0 || s[i] % 8 != 0 || s[i] >= (1ll << 38))) return false;
    return reinterpret_cast<uintptr_t>(r.p) % 16 == 0;
}

bool la_tc_together(const LaSweep &x, const LaSweep &y) {
    return (x.dk <= 64) == (y.dk <= 64) && (x.dv <= 64) == (y.dv <= 64) && x.n_seg == y.n_seg && x.seg == y.seg;
}

}  // namespace pararnn
