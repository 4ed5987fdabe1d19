// layers_api.cu -- C entry points of the sequence-layer operators: linear attention with a decay for each head
// (chunked form, backward pass, single-token step) and group norm with an activation or a gate.
#include <cmath>

#include "group_norm.cuh"
#include "linear_attention.cuh"

namespace pararnn {
namespace {

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Extent {  // bytes [p, p + n) that a call touches
    const void *p;
    size_t n;
};
bool overlaps(const Extent &a, const Extent &b) {
    const auto pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    return a.n && b.n && a.p && b.p && pa < pb + b.n && pb < pa + a.n;
}
// no output overlaps another output or an input
bool disjoint(const Extent *out, int n_out, const Extent *in, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i], out[j])) return false;
        for (int j = 0; j < n_in; ++j)
            if (overlaps(out[i], in[j])) return false;
    }
    return true;
}

size_t esize(int dtype) { return dtype == PARARNN_F32 ? 4 : 2; }
bool dtype_ok(int d) { return d == PARARNN_F32 || d == PARARNN_BF16; }

bool shape_ok(const pararnn_attention_shape *s) {
    if (s == nullptr || s->B < 1 || s->T < 1 || s->H < 1 || s->Hkv < 1 || s->H % s->Hkv != 0) return false;
    if (s->dk < 1 || s->dk > 128 || s->dv < 1 || s->dv > 128 || !dtype_ok(s->dtype)) return false;
    if (!std::isfinite(s->scale)) return false;
    // CTAs are counted in 32 bits: up to 64 per row and head
    return static_cast<long long>(s->B) * s->H <= (1ll << 24);
}

// An operand [B, T, heads, width]: aligned to its elements, strides that address forward.
bool rows_ok(const pararnn_rows *r, int dtype) {
    return r != nullptr && r->ptr != nullptr && aligned(r->ptr, esize(dtype)) && r->stride_b >= 0 && r->stride_t >= 0 &&
           r->stride_h >= 0;
}
Extent extent(const pararnn_rows &r, long long B, long long T, long long heads, long long width, int dtype) {
    const size_t last = (B - 1) * r.stride_b + (T - 1) * r.stride_t + (heads - 1) * r.stride_h + width;
    return {r.ptr, last * esize(dtype)};
}
LaRows operand(const pararnn_rows &r, int group) { return {r.ptr, r.stride_b, r.stride_t, r.stride_h, group}; }
LaRows dense(const void *p, long long T, long long heads, long long width, int group) {
    return {p, T * heads * width, heads * width, width, group};
}

size_t state_bytes(const pararnn_attention_shape &s) { return static_cast<size_t>(s.B) * s.H * s.dk * s.dv * 4; }
size_t seg_bytes(const pararnn_attention_shape &s, const LaPlan &p) {
    return p.n_seg > 1 ? align256(state_bytes(s) * p.n_seg) : 0;
}
// fp32 partial gradients [B, T, H, width] of each head where keys and values are shared
size_t part_bytes(const pararnn_attention_shape &s, int width) {
    return s.H == s.Hkv ? 0 : align256(static_cast<size_t>(s.B) * s.T * s.H * width * sizeof(float));
}

LaSweep sweep_of(const pararnn_attention_shape &s, const float *log_decay, const int *lengths, int dk, int dv) {
    LaSweep w{};
    w.B = s.B, w.T = s.T, w.H = s.H, w.dk = dk, w.dv = dv, w.dtype = s.dtype;
    w.log_decay = log_decay;
    w.lengths = lengths;
    return w;
}
void set_plan(LaSweep &w, const LaPlan &p, void *seg_state) {
    w.n_seg = p.n_seg, w.seg = p.seg;
    w.seg_state = static_cast<float *>(seg_state);
}

}  // namespace
}  // namespace pararnn

using namespace pararnn;

extern "C" {

size_t pararnn_linear_attention_workspace_size(const pararnn_attention_shape *shape) {
    if (!shape_ok(shape)) return 0;
    const pararnn_attention_shape &s = *shape;
    const size_t n = seg_bytes(s, la_plan(s.B, s.T, s.H, s.dk, s.dv, s.dtype));
    return n ? n : 256;
}

int pararnn_linear_attention(const pararnn_attention_shape *shape, const pararnn_rows *q, const pararnn_rows *k,
                             const pararnn_rows *v, const float *log_decay, const float *s0, const int *lengths,
                             void *o, float *s_out, void *workspace, size_t ws_bytes, pararnn_stream stream) {
    const size_t need = pararnn_linear_attention_workspace_size(shape);
    if (need == 0 || ws_bytes < need || !workspace || !aligned(workspace, 256)) return PARARNN_INVALID_ARG;
    const pararnn_attention_shape &s = *shape;
    if (!rows_ok(q, s.dtype) || !rows_ok(k, s.dtype) || !rows_ok(v, s.dtype)) return PARARNN_INVALID_ARG;
    if (!log_decay || !aligned(log_decay, 4) || !aligned(s0, 16) || !aligned(lengths, 4) || !o || !aligned(o, 16) ||
        !s_out || !aligned(s_out, 16))
        return PARARNN_INVALID_ARG;
    const Extent out[] = {{o, static_cast<size_t>(s.B) * s.T * s.H * s.dv * esize(s.dtype)},
                          {s_out, state_bytes(s)},
                          {workspace, need}};
    const Extent in[] = {extent(*q, s.B, s.T, s.H, s.dk, s.dtype), extent(*k, s.B, s.T, s.Hkv, s.dk, s.dtype),
                         extent(*v, s.B, s.T, s.Hkv, s.dv, s.dtype), {log_decay, s.H * sizeof(float)},
                         {lengths, s.B * sizeof(int)}, {s0 == s_out ? nullptr : s0, state_bytes(s)}};
    if (!disjoint(out, 3, in, 6)) return PARARNN_INVALID_ARG;
    LaSweep w = sweep_of(s, log_decay, lengths, s.dk, s.dv);
    w.a = operand(*q, 1), w.b = operand(*k, s.H / s.Hkv), w.c = operand(*v, s.H / s.Hkv);
    w.s_in = s0, w.s_out = s_out, w.s_i = s.dv, w.s_j = 1;
    w.out = o;
    w.e = 1;
    w.intra = w.inter = s.scale, w.update = 1.f;
    set_plan(w, la_plan(s.B, s.T, s.H, s.dk, s.dv, s.dtype), workspace);
    return launch_la_sweeps(&w, 1, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PARARNN_OK : PARARNN_CUDA_ERROR;
}

size_t pararnn_linear_attention_backward_workspace_size(const pararnn_attention_shape *shape) {
    if (!shape_ok(shape)) return 0;
    const pararnn_attention_shape &s = *shape;
    // three sweeps that may run at once; those for dq and dk swap the roles of the widths
    const size_t n = seg_bytes(s, la_plan(s.B, s.T, s.H, s.dk, s.dv, s.dtype)) +
                     2 * seg_bytes(s, la_plan(s.B, s.T, s.H, s.dv, s.dk, s.dtype)) + part_bytes(s, s.dk) +
                     part_bytes(s, s.dv);
    return n ? n : 256;
}

int pararnn_linear_attention_backward(const pararnn_attention_shape *shape, const pararnn_rows *q,
                                      const pararnn_rows *k, const pararnn_rows *v, const float *log_decay,
                                      const pararnn_rows *d_o, const float *s0, const float *ds, const int *lengths,
                                      void *dq, void *dk, void *dv, float *ds0, void *workspace, size_t ws_bytes,
                                      pararnn_stream stream) {
    const size_t need = pararnn_linear_attention_backward_workspace_size(shape);
    if (need == 0 || ws_bytes < need || !workspace || !aligned(workspace, 256)) return PARARNN_INVALID_ARG;
    const pararnn_attention_shape &s = *shape;
    if (!rows_ok(q, s.dtype) || !rows_ok(k, s.dtype) || !rows_ok(v, s.dtype) || !rows_ok(d_o, s.dtype))
        return PARARNN_INVALID_ARG;
    if (!log_decay || !aligned(log_decay, 4) || !aligned(s0, 16) || !aligned(ds, 16) || !aligned(lengths, 4) || !dq ||
        !dk || !dv || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(ds0, 16))
        return PARARNN_INVALID_ARG;
    const size_t rows = static_cast<size_t>(s.B) * s.T, e = esize(s.dtype);
    const Extent out[] = {{dq, rows * s.H * s.dk * e},
                          {dk, rows * s.Hkv * s.dk * e},
                          {dv, rows * s.Hkv * s.dv * e},
                          {ds0, state_bytes(s)},
                          {workspace, need}};
    const Extent in[] = {extent(*q, s.B, s.T, s.H, s.dk, s.dtype),   extent(*k, s.B, s.T, s.Hkv, s.dk, s.dtype),
                         extent(*v, s.B, s.T, s.Hkv, s.dv, s.dtype), extent(*d_o, s.B, s.T, s.H, s.dv, s.dtype),
                         {log_decay, s.H * sizeof(float)},           {lengths, s.B * sizeof(int)},
                         {s0, state_bytes(s)},                       {ds, state_bytes(s)}};
    if (!disjoint(out, 5, in, 8)) return PARARNN_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int per = s.H / s.Hkv;
    const LaPlan plan_v = la_plan(s.B, s.T, s.H, s.dk, s.dv, s.dtype);  // the sweep whose state is [dk, dv]
    const LaPlan plan_k = la_plan(s.B, s.T, s.H, s.dv, s.dk, s.dtype);  // the sweeps whose state is [dv, dk]
    char *at = static_cast<char *>(workspace);
    auto take = [&](size_t n) {
        char *p = at;
        at += n;
        return p;
    };
    float *part_k = reinterpret_cast<float *>(take(part_bytes(s, s.dk)));
    float *part_v = reinterpret_cast<float *>(take(part_bytes(s, s.dv)));
    LaSweep w[3];

    // dq: the forward sweep on (do, v, k) from S_0^T
    w[0] = sweep_of(s, log_decay, lengths, s.dv, s.dk);
    w[0].a = operand(*d_o, 1), w[0].b = operand(*v, per), w[0].c = operand(*k, per);
    w[0].s_in = s0, w[0].s_i = 1, w[0].s_j = s.dv;
    w[0].out = dq;
    w[0].e = 1;
    w[0].intra = w[0].inter = s.scale, w[0].update = 1.f;
    set_plan(w[0], plan_k, take(seg_bytes(s, plan_k)));

    // dk: the reversed sweep on (v, do, q) from dS^T
    w[1] = sweep_of(s, log_decay, lengths, s.dv, s.dk);
    w[1].a = operand(*v, per), w[1].b = operand(*d_o, 1), w[1].c = operand(*q, 1);
    w[1].s_in = ds, w[1].s_i = 1, w[1].s_j = s.dv;
    w[1].out = per == 1 ? dk : part_k;
    w[1].out_f32 = per != 1;
    w[1].reverse = 1;
    w[1].intra = w[1].update = s.scale, w[1].inter = 1.f;
    set_plan(w[1], plan_k, take(seg_bytes(s, plan_k)));

    // dv: the reversed sweep on (k, q, do) from dS; its last state is dL/dS_0
    w[2] = sweep_of(s, log_decay, lengths, s.dk, s.dv);
    w[2].a = operand(*k, per), w[2].b = operand(*q, 1), w[2].c = operand(*d_o, 1);
    w[2].s_in = ds, w[2].s_out = ds0, w[2].s_i = s.dv, w[2].s_j = 1;
    w[2].out = per == 1 ? dv : part_v;
    w[2].out_f32 = per != 1;
    w[2].reverse = 1;
    w[2].intra = w[2].update = s.scale, w[2].inter = 1.f;
    set_plan(w[2], plan_v, take(seg_bytes(s, plan_v)));

    if (launch_la_sweeps(w, 3, st) != cudaSuccess) return PARARNN_CUDA_ERROR;
    const long long n = static_cast<long long>(rows);
    if (per != 1 && (launch_la_group_sum(part_k, dk, s.dtype, n, s.Hkv, per, s.dk, st) != cudaSuccess ||
                     launch_la_group_sum(part_v, dv, s.dtype, n, s.Hkv, per, s.dv, st) != cudaSuccess))
        return PARARNN_CUDA_ERROR;
    return PARARNN_OK;
}

int pararnn_linear_attention_step(const pararnn_attention_shape *shape, const pararnn_rows *q, const pararnn_rows *k,
                                  const pararnn_rows *v, const float *log_decay, const float *state, const int *slots,
                                  int n_slots, void *o, float *out_state, pararnn_stream stream) {
    if (!shape_ok(shape) || shape->T != 1 || n_slots < 1) return PARARNN_INVALID_ARG;
    const pararnn_attention_shape &s = *shape;
    if (!rows_ok(q, s.dtype) || !rows_ok(k, s.dtype) || !rows_ok(v, s.dtype)) return PARARNN_INVALID_ARG;
    if (!slots && n_slots != s.B) return PARARNN_INVALID_ARG;
    if (!log_decay || !aligned(log_decay, 4) || !state || !aligned(state, 16) || !aligned(slots, 4) || !o ||
        !aligned(o, 16) || !out_state || !aligned(out_state, 16))
        return PARARNN_INVALID_ARG;
    const size_t pool = static_cast<size_t>(n_slots) * s.H * s.dk * s.dv * 4;
    const Extent out[] = {{o, static_cast<size_t>(s.B) * s.H * s.dv * esize(s.dtype)}, {out_state, pool}};
    const Extent in[] = {extent(*q, s.B, 1, s.H, s.dk, s.dtype), extent(*k, s.B, 1, s.Hkv, s.dk, s.dtype),
                         extent(*v, s.B, 1, s.Hkv, s.dv, s.dtype), {log_decay, s.H * sizeof(float)},
                         {slots, s.B * sizeof(int)}, {state == out_state ? nullptr : state, pool}};
    if (!disjoint(out, 2, in, 6)) return PARARNN_INVALID_ARG;
    LaStep w{};
    w.B = s.B, w.H = s.H, w.dk = s.dk, w.dv = s.dv, w.dtype = s.dtype, w.n_slots = n_slots;
    w.q = operand(*q, 1), w.k = operand(*k, s.H / s.Hkv), w.v = operand(*v, s.H / s.Hkv);
    w.log_decay = log_decay, w.state = state, w.slots = slots, w.scale = s.scale;
    w.out = o, w.out_state = out_state;
    return launch_la_step(w, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PARARNN_OK : PARARNN_CUDA_ERROR;
}

// ---- group norm ----------------------------------------------------------------------------------------------

static bool norm_ok(const pararnn_norm_shape *s) {
    if (s == nullptr || s->N < 1 || s->S < 1 || s->C < 1 || s->groups < 1 || s->C % s->groups != 0) return false;
    if (s->groups > 2048 || !dtype_ok(s->x_dtype) || !dtype_ok(s->y_dtype)) return false;
    if (s->act < PARARNN_ACT_NONE || s->act > PARARNN_ACT_GELU) return false;
    if (!std::isfinite(s->eps) || s->eps < 0.f) return false;
    // blocks of rows are counted in 32 bits: at most one per row
    return static_cast<long long>(s->N) * s->S <= (1ll << 31) - 1;
}

static GnArgs norm_args(const pararnn_norm_shape &s) {
    GnArgs a{};
    a.N = s.N, a.S = s.S, a.C = s.C, a.G = s.groups, a.x_dtype = s.x_dtype, a.y_dtype = s.y_dtype;
    a.act = s.act, a.eps = s.eps;
    return a;
}

size_t pararnn_group_norm_workspace_size(const pararnn_norm_shape *shape) {
    return norm_ok(shape) ? gn_ws_bytes(norm_args(*shape), false) : 0;
}

size_t pararnn_group_norm_backward_workspace_size(const pararnn_norm_shape *shape) {
    return norm_ok(shape) ? gn_ws_bytes(norm_args(*shape), true) : 0;
}

int pararnn_group_norm(const pararnn_norm_shape *shape, const void *x, const float *weight, const float *bias,
                       const void *gate, const int *lengths, void *y, float *stats, void *workspace, size_t ws_bytes,
                       pararnn_stream stream) {
    const size_t need = pararnn_group_norm_workspace_size(shape);
    if (need == 0 || ws_bytes < need || !workspace || !aligned(workspace, 256)) return PARARNN_INVALID_ARG;
    const pararnn_norm_shape &s = *shape;
    if (!x || !y || !stats || !aligned(x, 16) || !aligned(y, 16) || !aligned(stats, 16) || !aligned(weight, 16) ||
        !aligned(bias, 16) || !aligned(gate, 16) || !aligned(lengths, 4))
        return PARARNN_INVALID_ARG;
    const size_t n = static_cast<size_t>(s.N) * s.S * s.C;
    const Extent out[] = {{y, n * esize(s.y_dtype)}, {stats, static_cast<size_t>(s.N) * s.groups * 8}, {workspace, need}};
    const Extent in[] = {{x, n * esize(s.x_dtype)}, {gate, n * esize(s.x_dtype)}, {weight, s.C * sizeof(float)},
                         {bias, s.C * sizeof(float)}, {lengths, s.N * sizeof(int)}};
    if (!disjoint(out, 3, in, 5)) return PARARNN_INVALID_ARG;
    GnArgs a = norm_args(s);
    a.x = x, a.weight = weight, a.bias = bias, a.gate = gate, a.lengths = lengths, a.y = y, a.stats = stats;
    a.ws = static_cast<char *>(workspace);
    return launch_gn_forward(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PARARNN_OK : PARARNN_CUDA_ERROR;
}

int pararnn_group_norm_backward(const pararnn_norm_shape *shape, const void *x, const float *stats, const void *dy,
                                const float *weight, const float *bias, const void *gate, const int *lengths, void *dx,
                                float *dweight, float *dbias, void *dgate, void *workspace, size_t ws_bytes,
                                pararnn_stream stream) {
    const size_t need = pararnn_group_norm_backward_workspace_size(shape);
    if (need == 0 || ws_bytes < need || !workspace || !aligned(workspace, 256)) return PARARNN_INVALID_ARG;
    const pararnn_norm_shape &s = *shape;
    if (!x || !stats || !dy || !dx || !aligned(x, 16) || !aligned(dy, 16) || !aligned(dx, 16) || !aligned(stats, 16) ||
        !aligned(weight, 16) || !aligned(bias, 16) || !aligned(gate, 16) || !aligned(dgate, 16) ||
        !aligned(dweight, 16) || !aligned(dbias, 16) || !aligned(lengths, 4))
        return PARARNN_INVALID_ARG;
    if ((gate == nullptr) != (dgate == nullptr)) return PARARNN_INVALID_ARG;
    const size_t n = static_cast<size_t>(s.N) * s.S * s.C, par = s.C * sizeof(float);
    const Extent out[] = {{dx, n * esize(s.x_dtype)}, {dgate, n * esize(s.x_dtype)}, {dweight, par}, {dbias, par},
                          {workspace, need}};
    const Extent in[] = {{x, n * esize(s.x_dtype)}, {gate, n * esize(s.x_dtype)}, {dy, n * esize(s.y_dtype)},
                         {stats, static_cast<size_t>(s.N) * s.groups * 8}, {weight, par}, {bias, par},
                         {lengths, s.N * sizeof(int)}};
    if (!disjoint(out, 5, in, 7)) return PARARNN_INVALID_ARG;
    GnArgs a = norm_args(s);
    a.x = x, a.weight = weight, a.bias = bias, a.gate = gate, a.lengths = lengths;
    a.stats = const_cast<float *>(stats), a.y = const_cast<void *>(dy);
    a.dx = dx, a.dgate = dgate, a.dweight = dweight, a.dbias = dbias;
    a.ws = static_cast<char *>(workspace);
    return launch_gn_backward(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PARARNN_OK
                                                                                       : PARARNN_CUDA_ERROR;
}

}  // extern "C"
