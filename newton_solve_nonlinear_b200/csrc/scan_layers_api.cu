// scan_layers_api.cu -- C entry points of the selective state space block: its scan, its short causal convolution and the
// norm of its residual stream.
#include <algorithm>
#include <cmath>

#include "api_checks.cuh"
#include "causal_conv.cuh"
#include "layer_norm.cuh"
#include "selective_scan.cuh"

namespace pararnn {
namespace {

// ---- selective scan ------------------------------------------------------------------------------------------

bool scan_ok(const pararnn_scan_shape *s) {
    if (s == nullptr || s->B < 1 || s->T < 1 || s->D < 1 || s->G < 1 || s->D % s->G != 0) return false;
    if (s->N < 1 || s->N > 64 || !dtype_ok(s->dtype) || (s->softplus != 0 && s->softplus != 1)) return false;
    if (s->T > 1 << 30) return false;  // tokens are counted in 32 bits, in chunks that may pass the end
    // CTAs are counted in 32 bits: at most one per channel and 64 of them per sequence and segment
    return static_cast<long long>(s->B) * s->D <= (1ll << 30);
}

SsRows operand(const pararnn_rows *r) {
    return r == nullptr ? SsRows{nullptr, 0, 0, 0} : SsRows{r->ptr, r->stride_b, r->stride_t, r->stride_h};
}

struct ScanCall {
    const pararnn_scan_shape &s;
    SsArgs a{};
    Carve ws;
    ScanCall(const pararnn_scan_shape &shape, void *workspace) : s(shape), ws{static_cast<char *>(workspace), 0} {
        a.B = s.B, a.T = s.T, a.D = s.D, a.G = s.G, a.N = s.N, a.dtype = s.dtype, a.softplus = s.softplus;
    }
    float *floats(size_t n) { return reinterpret_cast<float *>(ws.take(n * sizeof(float))); }
    size_t states() const { return static_cast<size_t>(s.B) * s.D * s.N; }
    size_t tokens() const { return static_cast<size_t>(s.B) * s.T; }
    size_t kept() const { return static_cast<size_t>((s.T + kSsKeep - 1) / kSsKeep) * states(); }
    void forward() {
        const SsPlan p = ss_plan(a);
        a.n_seg = p.n_seg, a.seg = p.seg;
        if (a.n_seg > 1) {
            a.seg_state = floats(a.n_seg * states());
            a.seg_dt = floats(static_cast<size_t>(a.n_seg) * s.B * s.D);
        }
    }
    void backward(bool has_kept) {
        forward();
        if (a.n_seg > 1) a.rev_state = floats(a.n_seg * states());
        if (!has_kept) a.kept = floats(kept());
        const size_t part = static_cast<size_t>(ss_backward_tiles(a)) * tokens() * s.G * s.N;
        a.part_b = floats(part), a.part_c = floats(part);
        a.part_a = floats(static_cast<size_t>(a.n_seg) * s.B * s.D * (s.N + 2));
    }
};

struct ScanInputs {
    const pararnn_rows *x, *dt, *b, *c, *gate;
    const float *a, *skip, *dt_bias;
    bool ok(const pararnn_scan_shape &s) const {
        return rows_ok(x, s.dtype) && rows_ok(dt, s.dtype) && rows_ok(b, s.dtype) && rows_ok(c, s.dtype) &&
               (gate == nullptr || rows_ok(gate, s.dtype)) && a != nullptr && aligned(a, 4) && aligned(skip, 4) &&
               aligned(dt_bias, 4);
    }
    static constexpr int kExtents = 8;
    void extents(const pararnn_scan_shape &s, Extent *e) const {
        e[0] = extent(*x, s.B, s.T, 1, s.D, s.dtype), e[1] = extent(*dt, s.B, s.T, 1, s.D, s.dtype);
        e[2] = extent(*b, s.B, s.T, s.G, s.N, s.dtype), e[3] = extent(*c, s.B, s.T, s.G, s.N, s.dtype);
        e[4] = gate == nullptr ? Extent{nullptr, 0} : extent(*gate, s.B, s.T, 1, s.D, s.dtype);
        e[5] = {a, static_cast<size_t>(s.D) * s.N * 4}, e[6] = {skip, s.D * sizeof(float)};
        e[7] = {dt_bias, s.D * sizeof(float)};
    }
    template <typename Args>
    void to(Args &w) const {
        w.x = operand(x), w.dt = operand(dt), w.b = operand(b), w.c = operand(c), w.gate = operand(gate);
        w.a = a, w.skip = skip, w.dt_bias = dt_bias;
    }
};

// ---- causal convolution --------------------------------------------------------------------------------------

bool conv_ok(const pararnn_conv_shape *s) {
    if (s == nullptr || s->B < 1 || s->T < 1 || s->D < 1 || s->W < 2 || s->W > 8 || !dtype_ok(s->dtype)) return false;
    if (s->act != PARARNN_ACT_NONE && s->act != PARARNN_ACT_SILU) return false;
    if (s->T > 1 << 30) return false;  // tokens are counted in 32 bits, in runs that may pass the end
    return static_cast<long long>(s->B) * s->D <= (1ll << 30);  // CTAs are counted in 32 bits
}
CcArgs conv_args(const pararnn_conv_shape &s) {
    CcArgs a{};
    a.B = s.B, a.T = s.T, a.D = s.D, a.W = s.W, a.dtype = s.dtype, a.act = s.act;
    return a;
}
CcRows conv_rows(const pararnn_rows &r) { return {r.ptr, r.stride_b, r.stride_t}; }

// ---- the stream's norm ---------------------------------------------------------------------------------------

bool stream_ok(const pararnn_stream_shape *s) {
    if (s == nullptr || s->N < 1 || s->S < 1 || s->C < 1 || s->C > 1 << 30) return false;
    if (!dtype_ok(s->x_dtype) || !dtype_ok(s->r_dtype) || !dtype_ok(s->y_dtype) || (s->rms != 0 && s->rms != 1)) return false;
    if (!std::isfinite(s->eps) || s->eps < 0.f) return false;
    return static_cast<long long>(s->N) * s->S <= (1ll << 31) - 1;  // rows are counted in 32 bits
}
LnArgs stream_args(const pararnn_stream_shape &s) {
    LnArgs a{};
    a.N = s.N, a.S = s.S, a.C = s.C, a.x_dtype = s.x_dtype, a.r_dtype = s.r_dtype, a.y_dtype = s.y_dtype;
    a.rms = s.rms, a.eps = s.eps;
    return a;
}

int result(cudaError_t e) { return e == cudaSuccess ? PARARNN_OK : PARARNN_CUDA_ERROR; }

}  // namespace
}  // namespace pararnn

using namespace pararnn;

extern "C" {

size_t pararnn_selective_scan_workspace_size(const pararnn_scan_shape *shape) {
    if (!scan_ok(shape)) return 0;
    ScanCall c(*shape, nullptr);
    c.forward();
    return std::max(c.ws.used, kNone);
}

int pararnn_selective_scan(const pararnn_scan_shape *shape, const pararnn_rows *x, const pararnn_rows *dt, const float *a,
                           const pararnn_rows *b, const pararnn_rows *c, const float *skip, const pararnn_rows *gate,
                           const float *dt_bias, const float *h0, const int *lengths, void *y, float *h, float *kept,
                           void *workspace, size_t ws_bytes, pararnn_stream stream) {
    const size_t need = pararnn_selective_scan_workspace_size(shape);
    if (!workspace_ok(need, workspace, ws_bytes)) return PARARNN_INVALID_ARG;
    const pararnn_scan_shape &s = *shape;
    const ScanInputs in{x, dt, b, c, gate, a, skip, dt_bias};
    if (!in.ok(s) || !aligned(h0, 16) || !aligned(lengths, 4) || !y || !aligned(y, 16) || !h || !aligned(h, 16) ||
        !aligned(kept, 16))
        return PARARNN_INVALID_ARG;
    ScanCall call(s, workspace);
    const Extent outs[] = {{y, call.tokens() * s.D * esize(s.dtype)}, {h, call.states() * 4}, {kept, call.kept() * 4},
                           {workspace, need == kNone ? 0 : need}};
    Extent ins[ScanInputs::kExtents + 2];
    in.extents(s, ins);
    ins[ScanInputs::kExtents] = {lengths, s.B * sizeof(int)};
    ins[ScanInputs::kExtents + 1] = {h0 == h ? nullptr : h0, call.states() * 4};
    if (!disjoint(outs, 4, ins, ScanInputs::kExtents + 2)) return PARARNN_INVALID_ARG;
    call.forward();
    SsArgs &w = call.a;
    in.to(w);
    w.h0 = h0, w.lengths = lengths, w.y = y, w.h = h, w.kept = kept;
    return result(launch_ss_forward(w, reinterpret_cast<cudaStream_t>(stream)));
}

size_t pararnn_selective_scan_backward_workspace_size(const pararnn_scan_shape *shape, int has_kept) {
    if (!scan_ok(shape)) return 0;
    ScanCall c(*shape, nullptr);
    c.backward(has_kept != 0);
    return std::max(c.ws.used, kNone);
}

int pararnn_selective_scan_backward(const pararnn_scan_shape *shape, const pararnn_rows *x, const pararnn_rows *dt,
                                    const float *a, const pararnn_rows *b, const pararnn_rows *c, const float *skip,
                                    const pararnn_rows *gate, const float *dt_bias, const pararnn_rows *dy, const float *h0,
                                    const float *dh, const int *lengths, const float *kept, void *dx, void *ddt, float *da,
                                    void *db, void *dc, float *dskip, void *dgate, float *ddt_bias, float *dh0,
                                    void *workspace, size_t ws_bytes, pararnn_stream stream) {
    const size_t need = pararnn_selective_scan_backward_workspace_size(shape, kept != nullptr);
    if (!workspace_ok(need, workspace, ws_bytes)) return PARARNN_INVALID_ARG;
    const pararnn_scan_shape &s = *shape;
    const ScanInputs in{x, dt, b, c, gate, a, skip, dt_bias};
    if (!in.ok(s) || !rows_ok(dy, s.dtype) || !aligned(h0, 16) || !aligned(dh, 16) || !aligned(lengths, 4) ||
        !aligned(kept, 16))
        return PARARNN_INVALID_ARG;
    if (!dx || !ddt || !da || !db || !dc || (gate == nullptr) != (dgate == nullptr)) return PARARNN_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(dx), static_cast<const void *>(ddt), static_cast<const void *>(da),
                          static_cast<const void *>(db), static_cast<const void *>(dc), static_cast<const void *>(dskip),
                          static_cast<const void *>(dgate), static_cast<const void *>(ddt_bias),
                          static_cast<const void *>(dh0)})
        if (!aligned(p, 16)) return PARARNN_INVALID_ARG;
    ScanCall call(s, workspace);
    const size_t e = esize(s.dtype), rows = call.tokens() * s.D * e, shared = call.tokens() * s.G * s.N * e;
    const Extent outs[] = {{dx, rows}, {ddt, rows}, {da, static_cast<size_t>(s.D) * s.N * 4}, {db, shared}, {dc, shared},
                           {dskip, s.D * sizeof(float)}, {dgate, rows}, {ddt_bias, s.D * sizeof(float)},
                           {dh0, call.states() * 4}, {workspace, need == kNone ? 0 : need}};
    Extent ins[ScanInputs::kExtents + 5];
    in.extents(s, ins);
    Extent *more = ins + ScanInputs::kExtents;
    more[0] = extent(*dy, s.B, s.T, 1, s.D, s.dtype), more[1] = {lengths, s.B * sizeof(int)};
    more[2] = {h0, call.states() * 4}, more[3] = {dh, call.states() * 4}, more[4] = {kept, call.kept() * 4};
    if (!disjoint(outs, 10, ins, ScanInputs::kExtents + 5)) return PARARNN_INVALID_ARG;
    call.backward(kept != nullptr);
    SsArgs &w = call.a;
    in.to(w);
    w.dy = operand(dy);
    w.h0 = h0, w.dh = dh, w.lengths = lengths;
    w.dx = dx, w.ddt = ddt, w.da = da, w.db = db, w.dc = dc, w.dskip = dskip, w.dgate = dgate, w.ddt_bias = ddt_bias;
    w.dh0 = dh0;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (kept != nullptr) {
        w.kept = const_cast<float *>(kept);
    } else {
        const cudaError_t err = launch_ss_kept(w, st);
        if (err != cudaSuccess) return PARARNN_CUDA_ERROR;
    }
    return result(launch_ss_backward(w, st));
}

int pararnn_selective_scan_step(const pararnn_scan_shape *shape, const pararnn_rows *x, const pararnn_rows *dt,
                                const float *a, const pararnn_rows *b, const pararnn_rows *c, const float *skip,
                                const pararnn_rows *gate, const float *dt_bias, const float *state, const int *slots,
                                int n_slots, void *y, float *out_state, pararnn_stream stream) {
    if (!scan_ok(shape) || shape->T != 1 || n_slots < 1) return PARARNN_INVALID_ARG;
    const pararnn_scan_shape &s = *shape;
    const ScanInputs in{x, dt, b, c, gate, a, skip, dt_bias};
    if (!in.ok(s) || (!slots && n_slots != s.B)) return PARARNN_INVALID_ARG;
    if (!state || !aligned(state, 16) || !aligned(slots, 4) || !y || !aligned(y, 16) || !out_state || !aligned(out_state, 16))
        return PARARNN_INVALID_ARG;
    const size_t pool = static_cast<size_t>(n_slots) * s.D * s.N * 4;
    const Extent outs[] = {{y, static_cast<size_t>(s.B) * s.D * esize(s.dtype)}, {out_state, pool}};
    Extent ins[ScanInputs::kExtents + 2];
    in.extents(s, ins);
    ins[ScanInputs::kExtents] = {slots, s.B * sizeof(int)};
    ins[ScanInputs::kExtents + 1] = {state == out_state ? nullptr : state, pool};
    if (!disjoint(outs, 2, ins, ScanInputs::kExtents + 2)) return PARARNN_INVALID_ARG;
    SsStep w{};
    w.B = s.B, w.D = s.D, w.G = s.G, w.N = s.N, w.dtype = s.dtype, w.softplus = s.softplus, w.n_slots = n_slots;
    in.to(w);
    w.state = state, w.slots = slots, w.y = y, w.out_state = out_state;
    return result(launch_ss_step(w, reinterpret_cast<cudaStream_t>(stream)));
}

int pararnn_causal_conv(const pararnn_conv_shape *shape, const pararnn_rows *x, const float *weight, const float *bias,
                        const void *state, const int *lengths, void *y, void *last, pararnn_stream stream) {
    if (!conv_ok(shape) || !rows_ok(x, shape->dtype)) return PARARNN_INVALID_ARG;
    const pararnn_conv_shape &s = *shape;
    if (!weight || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(state, 16) || !aligned(lengths, 4) || !y ||
        !aligned(y, 16) || !last || !aligned(last, 16))
        return PARARNN_INVALID_ARG;
    const size_t e = esize(s.dtype), ends = static_cast<size_t>(s.B) * (s.W - 1) * s.D * e;
    const Extent outs[] = {{y, static_cast<size_t>(s.B) * s.T * s.D * e}, {last, ends}};
    const Extent ins[] = {extent(*x, s.B, s.T, 1, s.D, s.dtype), {weight, static_cast<size_t>(s.D) * s.W * 4},
                          {bias, s.D * sizeof(float)}, {state, ends}, {lengths, s.B * sizeof(int)}};
    if (!disjoint(outs, 2, ins, 5)) return PARARNN_INVALID_ARG;
    CcArgs a = conv_args(s);
    a.x = conv_rows(*x), a.weight = weight, a.bias = bias, a.state = state, a.lengths = lengths, a.y = y, a.last = last;
    return result(launch_cc_forward(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t pararnn_causal_conv_backward_workspace_size(const pararnn_conv_shape *shape) {
    if (!conv_ok(shape)) return 0;
    const pararnn_conv_shape &s = *shape;
    return align256(static_cast<size_t>(cc_backward_rows(conv_args(s))) * s.D * (s.W + 1) * sizeof(float));
}

int pararnn_causal_conv_backward(const pararnn_conv_shape *shape, const pararnn_rows *x, const float *weight,
                                 const float *bias, const pararnn_rows *dy, const void *state, const void *dlast,
                                 const int *lengths, void *dx, float *dweight, float *dbias, void *dstate, void *workspace,
                                 size_t ws_bytes, pararnn_stream stream) {
    const size_t need = pararnn_causal_conv_backward_workspace_size(shape);
    if (!workspace_ok(need, workspace, ws_bytes)) return PARARNN_INVALID_ARG;
    const pararnn_conv_shape &s = *shape;
    if (!rows_ok(x, s.dtype) || !rows_ok(dy, s.dtype) || !weight || !aligned(weight, 4) || !aligned(bias, 4) ||
        !aligned(state, 16) || !aligned(dlast, 16) || !aligned(lengths, 4) || !dx || !aligned(dx, 16) || !dweight ||
        !aligned(dweight, 16) || !aligned(dbias, 16) || !aligned(dstate, 16))
        return PARARNN_INVALID_ARG;
    const size_t e = esize(s.dtype), ends = static_cast<size_t>(s.B) * (s.W - 1) * s.D * e,
                 taps = static_cast<size_t>(s.D) * s.W * 4;
    const Extent outs[] = {{dx, static_cast<size_t>(s.B) * s.T * s.D * e}, {dweight, taps}, {dbias, s.D * sizeof(float)},
                           {dstate, ends}, {workspace, need}};
    const Extent ins[] = {extent(*x, s.B, s.T, 1, s.D, s.dtype), extent(*dy, s.B, s.T, 1, s.D, s.dtype), {weight, taps},
                          {bias, s.D * sizeof(float)}, {state, ends}, {dlast, ends}, {lengths, s.B * sizeof(int)}};
    if (!disjoint(outs, 5, ins, 7)) return PARARNN_INVALID_ARG;
    CcArgs a = conv_args(s);
    a.x = conv_rows(*x), a.dy = conv_rows(*dy), a.weight = weight, a.bias = bias, a.state = state, a.dlast = dlast;
    a.lengths = lengths, a.dx = dx, a.dweight = dweight, a.dbias = dbias, a.dstate = dstate;
    a.part = static_cast<float *>(workspace);
    return result(launch_cc_backward(a, reinterpret_cast<cudaStream_t>(stream)));
}

int pararnn_causal_conv_step(const pararnn_conv_shape *shape, const pararnn_rows *x, const float *weight, const float *bias,
                             const void *state, const int *slots, int n_slots, void *y, void *out_state,
                             pararnn_stream stream) {
    if (!conv_ok(shape) || shape->T != 1 || n_slots < 1 || !rows_ok(x, shape->dtype)) return PARARNN_INVALID_ARG;
    const pararnn_conv_shape &s = *shape;
    if (!slots && n_slots != s.B) return PARARNN_INVALID_ARG;
    if (!weight || !aligned(weight, 4) || !aligned(bias, 4) || !state || !aligned(state, 16) || !aligned(slots, 4) || !y ||
        !aligned(y, 16) || !out_state || !aligned(out_state, 16))
        return PARARNN_INVALID_ARG;
    const size_t e = esize(s.dtype), pool = static_cast<size_t>(n_slots) * (s.W - 1) * s.D * e;
    const Extent outs[] = {{y, static_cast<size_t>(s.B) * s.D * e}, {out_state, pool}};
    const Extent ins[] = {extent(*x, s.B, 1, 1, s.D, s.dtype), {weight, static_cast<size_t>(s.D) * s.W * 4},
                          {bias, s.D * sizeof(float)}, {slots, s.B * sizeof(int)},
                          {state == out_state ? nullptr : state, pool}};
    if (!disjoint(outs, 2, ins, 5)) return PARARNN_INVALID_ARG;
    CcStep w{};
    w.B = s.B, w.D = s.D, w.W = s.W, w.dtype = s.dtype, w.act = s.act, w.n_slots = n_slots;
    w.x = conv_rows(*x), w.weight = weight, w.bias = bias, w.state = state, w.slots = slots, w.y = y, w.out_state = out_state;
    return result(launch_cc_step(w, reinterpret_cast<cudaStream_t>(stream)));
}

int pararnn_layer_norm(const pararnn_stream_shape *shape, const void *x, const void *residual, const float *weight,
                       const float *bias, const int *lengths, void *y, void *r, float *stats, pararnn_stream stream) {
    if (!stream_ok(shape)) return PARARNN_INVALID_ARG;
    const pararnn_stream_shape &s = *shape;
    if (!x || !y || !stats || (residual == nullptr) != (r == nullptr)) return PARARNN_INVALID_ARG;
    for (const void *p : {x, residual, static_cast<const void *>(weight), static_cast<const void *>(bias),
                          static_cast<const void *>(y), static_cast<const void *>(r), static_cast<const void *>(stats)})
        if (!aligned(p, 16)) return PARARNN_INVALID_ARG;
    if (!aligned(lengths, 4)) return PARARNN_INVALID_ARG;
    const size_t rows = static_cast<size_t>(s.N) * s.S, n = rows * s.C, par = s.C * sizeof(float);
    const Extent outs[] = {{y, n * esize(s.y_dtype)}, {r, n * esize(s.r_dtype)}, {stats, rows * 8}};
    const Extent ins[] = {{x, n * esize(s.x_dtype)}, {residual == r ? nullptr : residual, n * esize(s.r_dtype)}, {weight, par},
                          {bias, par}, {lengths, s.N * sizeof(int)}};
    if (!disjoint(outs, 3, ins, 5)) return PARARNN_INVALID_ARG;
    LnArgs a = stream_args(s);
    a.x = x, a.residual = residual, a.weight = weight, a.bias = bias, a.lengths = lengths, a.y = y, a.r = r, a.stats = stats;
    return result(launch_ln_forward(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t pararnn_layer_norm_backward_workspace_size(const pararnn_stream_shape *shape) {
    if (!stream_ok(shape)) return 0;
    return align256(static_cast<size_t>(ln_backward_rows(stream_args(*shape))) * 2 * shape->C * sizeof(float));
}

int pararnn_layer_norm_backward(const pararnn_stream_shape *shape, const void *r, const float *stats, const void *dy,
                                const float *weight, const void *dr_in, const int *lengths, void *dr, void *dx,
                                float *dweight, float *dbias, void *workspace, size_t ws_bytes, pararnn_stream stream) {
    const size_t need = pararnn_layer_norm_backward_workspace_size(shape);
    if (!workspace_ok(need, workspace, ws_bytes)) return PARARNN_INVALID_ARG;
    const pararnn_stream_shape &s = *shape;
    if (!r || !stats || !dy || !dr) return PARARNN_INVALID_ARG;
    for (const void *p : {r, static_cast<const void *>(stats), dy, static_cast<const void *>(weight), dr_in,
                          static_cast<const void *>(dr), static_cast<const void *>(dx), static_cast<const void *>(dweight),
                          static_cast<const void *>(dbias)})
        if (!aligned(p, 16)) return PARARNN_INVALID_ARG;
    if (!aligned(lengths, 4)) return PARARNN_INVALID_ARG;
    const size_t rows = static_cast<size_t>(s.N) * s.S, n = rows * s.C, par = s.C * sizeof(float);
    const Extent outs[] = {{dr, n * esize(s.r_dtype)}, {dx, n * esize(s.x_dtype)}, {dweight, par}, {dbias, par},
                           {workspace, need}};
    const Extent ins[] = {{r, n * esize(s.r_dtype)}, {stats, rows * 8}, {dy, n * esize(s.y_dtype)}, {weight, par},
                          {dr_in == dr ? nullptr : dr_in, n * esize(s.r_dtype)}, {lengths, s.N * sizeof(int)}};
    if (!disjoint(outs, 5, ins, 6)) return PARARNN_INVALID_ARG;
    LnArgs a = stream_args(s);
    a.weight = weight, a.lengths = lengths, a.r = const_cast<void *>(r), a.y = const_cast<void *>(dy);
    a.stats = const_cast<float *>(stats), a.dr_in = dr_in, a.dr = dr, a.dx = dx, a.dweight = dweight, a.dbias = dbias;
    a.part = static_cast<float *>(workspace);
    return result(launch_ln_backward(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
