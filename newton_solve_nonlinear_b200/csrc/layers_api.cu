// layers_api.cu -- C entry points of the sequence-layer operators: linear attention with a decay for each head
// (chunked form, backward pass, single-token step) and group norm with an activation or a gate.
#include <algorithm>
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

// What the size queries answer where a call needs no workspace: it then takes NULL.
constexpr size_t kNone = 1;
bool workspace_ok(size_t need, const void *p, size_t bytes) {
    return need == kNone || (need != 0 && p != nullptr && aligned(p, 256) && bytes >= need);
}

size_t esize(int dtype) { return dtype == PARARNN_F32 ? 4 : 2; }
bool dtype_ok(int d) { return d == PARARNN_F32 || d == PARARNN_BF16; }

bool shape_ok(const pararnn_attention_shape *s) {
    if (s == nullptr || s->B < 1 || s->T < 1 || s->H < 1 || s->Hkv < 1 || s->H % s->Hkv != 0) return false;
    if (s->dk < 1 || s->dk > 128 || s->dv < 1 || s->dv > 128 || !dtype_ok(s->dtype)) return false;
    if (!std::isfinite(s->scale)) return false;
    if (s->T > 1 << 30) return false;  // tokens are counted in 32 bits, in chunks that may pass the end
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

size_t state_bytes(const pararnn_attention_shape &s) { return static_cast<size_t>(s.B) * s.H * s.dk * s.dv * 4; }
int padded(int width) { return (width + 7) / 8 * 8; }

// Lays a call's workspace out; with no base it only counts.
struct Carve {
    char *base;
    size_t used;
    char *take(size_t n) {
        char *p = base + used;
        used += align256(n);
        return p;
    }
};

// The sweeps of a call, and what is packed before and unpacked after them.  Built the same way for the size query
// and for the call.
struct Call {
    const pararnn_attention_shape &s;
    Carve ws;
    LaSweep w[3];
    struct {
        LaRows from;
        void *to;
        int heads, width;
    } pack[4];
    struct {
        const void *from;
        void *to;
        int heads, width;
    } unpack[3];
    int n_pack = 0, n_unpack = 0;

    Call(const pararnn_attention_shape &shape, void *workspace)
        : s(shape), ws{static_cast<char *>(workspace), 0}, w{}, pack{}, unpack{} {}

    // bf16 rows come by TMA: those that it cannot read are packed first
    LaRows in(const pararnn_rows &r, int heads, int width) {
        const LaRows x = operand(r, s.H / heads);
        if (s.dtype != PARARNN_BF16 || la_tc_readable(x, s.B, s.T, heads)) return x;
        const int wp = padded(width);
        void *to = ws.take(static_cast<size_t>(s.B) * s.T * heads * wp * 2);
        pack[n_pack++] = {x, to, heads, width};
        return {to, static_cast<long long>(s.T) * heads * wp, static_cast<long long>(heads) * wp, wp, x.group};
    }
    // outputs of w [B, T, H, width]; bf16 rows leave by TMA, in rows of whole 16 bytes
    void out(LaSweep &x, void *p, int width) {
        x.out = p;
        x.out_w = width;
        if (s.dtype != PARARNN_BF16 || width % 8 == 0) return;
        x.out_w = padded(width);
        x.out = ws.take(static_cast<size_t>(s.B) * s.T * s.H * x.out_w * 2);
        unpack[n_unpack++] = {x.out, p, s.H, width};
    }
    // fp32 partial outputs of each head, where keys and values are shared
    float *partial(LaSweep &x, int width) {
        x.out_w = padded(width);
        x.out_f32 = 1;
        x.out = ws.take(static_cast<size_t>(s.B) * s.T * s.H * x.out_w * sizeof(float));
        return static_cast<float *>(x.out);
    }
    void sweep(LaSweep &x, const float *log_decay, const int *lengths, int dk, int dv, const LaPlan &p) {
        x.B = s.B, x.T = s.T, x.H = s.H, x.dk = dk, x.dv = dv, x.dtype = s.dtype;
        x.log_decay = log_decay, x.lengths = lengths;
        x.n_seg = p.n_seg, x.seg = p.seg;
        if (p.n_seg > 1) x.seg_state = reinterpret_cast<float *>(ws.take(state_bytes(s) * p.n_seg));
    }
    bool before(cudaStream_t st) const {
        for (int i = 0; i < n_pack; ++i)
            if (launch_la_pack(pack[i].from, pack[i].to, s.B, s.T, pack[i].heads, pack[i].width, st) != cudaSuccess)
                return false;
        return true;
    }
    bool after(cudaStream_t st) const {
        for (int i = 0; i < n_unpack; ++i)
            if (launch_la_unpack(unpack[i].from, unpack[i].to, static_cast<long long>(s.B) * s.T * unpack[i].heads,
                                 unpack[i].width, st) != cudaSuccess)
                return false;
        return true;
    }
};

void build_forward(Call &c, const pararnn_rows &q, const pararnn_rows &k, const pararnn_rows &v, const float *log_decay,
                   const float *s0, const int *lengths, void *o, float *s_out) {
    const pararnn_attention_shape &s = c.s;
    LaSweep &w = c.w[0];
    c.sweep(w, log_decay, lengths, s.dk, s.dv, la_plan(s.B, s.T, s.H, s.dk, s.dv, s.dtype, 1, lengths != nullptr));
    w.a = c.in(q, s.H, s.dk), w.b = c.in(k, s.Hkv, s.dk), w.c = c.in(v, s.Hkv, s.dv);
    w.s_in = s0, w.s_out = s_out, w.s_i = s.dv, w.s_j = 1;
    c.out(w, o, s.dv);
    w.e = 1;
    w.intra = w.inter = s.scale, w.update = 1.f;
}

struct Partials {
    float *k, *v;
};
Partials build_backward(Call &c, const pararnn_rows &q, const pararnn_rows &k, const pararnn_rows &v,
                        const float *log_decay, const pararnn_rows &d_o, const float *s0, const float *ds,
                        const int *lengths, void *dq, void *dk, void *dv, float *ds0) {
    const pararnn_attention_shape &s = c.s;
    const bool shared = s.H != s.Hkv;
    Partials part{};
    const LaRows rq = c.in(q, s.H, s.dk), rk = c.in(k, s.Hkv, s.dk), rv = c.in(v, s.Hkv, s.dv),
                 ro = c.in(d_o, s.H, s.dv);
    // of the sweep whose state is [dk, dv], and of the two whose state is [dv, dk]
    const LaPlan plan_v = la_plan(s.B, s.T, s.H, s.dk, s.dv, s.dtype, 3, lengths != nullptr);
    const LaPlan plan_k = la_plan(s.B, s.T, s.H, s.dv, s.dk, s.dtype, 3, lengths != nullptr);

    // dq: the forward sweep on (do, v, k) from S_0^T
    LaSweep &x = c.w[0];
    c.sweep(x, log_decay, lengths, s.dv, s.dk, plan_k);
    x.a = ro, x.b = rv, x.c = rk;
    x.s_in = s0, x.s_i = 1, x.s_j = s.dv;
    c.out(x, dq, s.dk);
    x.e = 1;
    x.intra = x.inter = s.scale, x.update = 1.f;

    // dk: the reversed sweep on (v, do, q) from dS^T
    LaSweep &y = c.w[1];
    c.sweep(y, log_decay, lengths, s.dv, s.dk, plan_k);
    y.a = rv, y.b = ro, y.c = rq;
    y.s_in = ds, y.s_i = 1, y.s_j = s.dv;
    if (shared) part.k = c.partial(y, s.dk);
    else c.out(y, dk, s.dk);
    y.reverse = 1;
    y.intra = y.update = s.scale, y.inter = 1.f;

    // dv: the reversed sweep on (k, q, do) from dS; its last state is dL/dS_0
    LaSweep &z = c.w[2];
    c.sweep(z, log_decay, lengths, s.dk, s.dv, plan_v);
    z.a = rk, z.b = rq, z.c = ro;
    z.s_in = ds, z.s_out = ds0, z.s_i = s.dv, z.s_j = 1;
    if (shared) part.v = c.partial(z, s.dv);
    else c.out(z, dv, s.dv);
    z.reverse = 1;
    z.intra = z.update = s.scale, z.inter = 1.f;
    return part;
}

}  // namespace
}  // namespace pararnn

using namespace pararnn;

extern "C" {

size_t pararnn_linear_attention_workspace_size(const pararnn_attention_shape *shape, const pararnn_rows *q,
                                               const pararnn_rows *k, const pararnn_rows *v) {
    if (!shape_ok(shape) || !rows_ok(q, shape->dtype) || !rows_ok(k, shape->dtype) || !rows_ok(v, shape->dtype)) return 0;
    size_t most = kNone;
    const int some = 0;
    for (const int *lengths : {static_cast<const int *>(nullptr), &some}) {  // with lengths or without: the larger
        Call c(*shape, nullptr);
        build_forward(c, *q, *k, *v, nullptr, nullptr, lengths, nullptr, nullptr);
        most = c.ws.used > most ? c.ws.used : most;
    }
    return most;
}

int pararnn_linear_attention(const pararnn_attention_shape *shape, const pararnn_rows *q, const pararnn_rows *k,
                             const pararnn_rows *v, const float *log_decay, const float *s0, const int *lengths,
                             void *o, float *s_out, void *workspace, size_t ws_bytes, pararnn_stream stream) {
    const size_t need = pararnn_linear_attention_workspace_size(shape, q, k, v);
    if (!workspace_ok(need, workspace, ws_bytes)) return PARARNN_INVALID_ARG;
    const pararnn_attention_shape &s = *shape;
    if (!log_decay || !aligned(log_decay, 4) || !aligned(s0, 16) || !aligned(lengths, 4) || !o || !aligned(o, 16) ||
        !s_out || !aligned(s_out, 16))
        return PARARNN_INVALID_ARG;
    const Extent out[] = {{o, static_cast<size_t>(s.B) * s.T * s.H * s.dv * esize(s.dtype)},
                          {s_out, state_bytes(s)},
                          {workspace, need == kNone ? 0 : need}};
    const Extent in[] = {extent(*q, s.B, s.T, s.H, s.dk, s.dtype), extent(*k, s.B, s.T, s.Hkv, s.dk, s.dtype),
                         extent(*v, s.B, s.T, s.Hkv, s.dv, s.dtype), {log_decay, s.H * sizeof(float)},
                         {lengths, s.B * sizeof(int)}, {s0 == s_out ? nullptr : s0, state_bytes(s)}};
    if (!disjoint(out, 3, in, 6)) return PARARNN_INVALID_ARG;
    Call c(s, workspace);
    build_forward(c, *q, *k, *v, log_decay, s0, lengths, o, s_out);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return c.before(st) && launch_la_sweeps(c.w, 1, st) == cudaSuccess && c.after(st) ? PARARNN_OK : PARARNN_CUDA_ERROR;
}

size_t pararnn_linear_attention_backward_workspace_size(const pararnn_attention_shape *shape, const pararnn_rows *q,
                                                        const pararnn_rows *k, const pararnn_rows *v,
                                                        const pararnn_rows *d_o) {
    if (!shape_ok(shape) || !rows_ok(q, shape->dtype) || !rows_ok(k, shape->dtype) || !rows_ok(v, shape->dtype) ||
        !rows_ok(d_o, shape->dtype))
        return 0;
    size_t most = kNone;
    const int some = 0;
    for (const int *lengths : {static_cast<const int *>(nullptr), &some}) {
        Call c(*shape, nullptr);
        build_backward(c, *q, *k, *v, nullptr, *d_o, nullptr, nullptr, lengths, nullptr, nullptr, nullptr, nullptr);
        most = c.ws.used > most ? c.ws.used : most;
    }
    return most;
}

int pararnn_linear_attention_backward(const pararnn_attention_shape *shape, const pararnn_rows *q,
                                      const pararnn_rows *k, const pararnn_rows *v, const float *log_decay,
                                      const pararnn_rows *d_o, const float *s0, const float *ds, const int *lengths,
                                      void *dq, void *dk, void *dv, float *ds0, void *workspace, size_t ws_bytes,
                                      pararnn_stream stream) {
    const size_t need = pararnn_linear_attention_backward_workspace_size(shape, q, k, v, d_o);
    if (!workspace_ok(need, workspace, ws_bytes)) return PARARNN_INVALID_ARG;
    const pararnn_attention_shape &s = *shape;
    if (!log_decay || !aligned(log_decay, 4) || !aligned(s0, 16) || !aligned(ds, 16) || !aligned(lengths, 4) || !dq ||
        !dk || !dv || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(ds0, 16))
        return PARARNN_INVALID_ARG;
    const size_t rows = static_cast<size_t>(s.B) * s.T, e = esize(s.dtype);
    const Extent out[] = {{dq, rows * s.H * s.dk * e},
                          {dk, rows * s.Hkv * s.dk * e},
                          {dv, rows * s.Hkv * s.dv * e},
                          {ds0, state_bytes(s)},
                          {workspace, need == kNone ? 0 : need}};
    const Extent in[] = {extent(*q, s.B, s.T, s.H, s.dk, s.dtype),   extent(*k, s.B, s.T, s.Hkv, s.dk, s.dtype),
                         extent(*v, s.B, s.T, s.Hkv, s.dv, s.dtype), extent(*d_o, s.B, s.T, s.H, s.dv, s.dtype),
                         {log_decay, s.H * sizeof(float)},           {lengths, s.B * sizeof(int)},
                         {s0, state_bytes(s)},                       {ds, state_bytes(s)}};
    if (!disjoint(out, 5, in, 8)) return PARARNN_INVALID_ARG;
    Call c(s, workspace);
    const Partials part = build_backward(c, *q, *k, *v, log_decay, *d_o, s0, ds, lengths, dq, dk, dv, ds0);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!c.before(st) || launch_la_sweeps(c.w, 3, st) != cudaSuccess || !c.after(st)) return PARARNN_CUDA_ERROR;
    const long long n = static_cast<long long>(rows);
    const int per = s.H / s.Hkv;
    if (per != 1 &&
        (launch_la_group_sum(part.k, dk, s.dtype, n, s.Hkv, per, s.dk, c.w[1].out_w, st) != cudaSuccess ||
         launch_la_group_sum(part.v, dv, s.dtype, n, s.Hkv, per, s.dv, c.w[2].out_w, st) != cudaSuccess))
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
    if (s->C > 1 << 30) return false;  // channels are counted in 32 bits, twice over and in steps past the end
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
    return norm_ok(shape) ? std::max(gn_ws_bytes(norm_args(*shape), false), kNone) : 0;
}

size_t pararnn_group_norm_backward_workspace_size(const pararnn_norm_shape *shape) {
    return norm_ok(shape) ? std::max(gn_ws_bytes(norm_args(*shape), true), kNone) : 0;
}

int pararnn_group_norm(const pararnn_norm_shape *shape, const void *x, const float *weight, const float *bias,
                       const void *gate, const int *lengths, void *y, float *stats, void *workspace, size_t ws_bytes,
                       pararnn_stream stream) {
    const size_t need = pararnn_group_norm_workspace_size(shape);
    if (!workspace_ok(need, workspace, ws_bytes)) return PARARNN_INVALID_ARG;
    const pararnn_norm_shape &s = *shape;
    if (!x || !y || !stats || !aligned(x, 16) || !aligned(y, 16) || !aligned(stats, 16) || !aligned(weight, 16) ||
        !aligned(bias, 16) || !aligned(gate, 16) || !aligned(lengths, 4))
        return PARARNN_INVALID_ARG;
    const size_t n = static_cast<size_t>(s.N) * s.S * s.C;
    const Extent out[] = {{y, n * esize(s.y_dtype)}, {stats, static_cast<size_t>(s.N) * s.groups * 8}, {workspace, need == kNone ? 0 : need}};
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
    if (!workspace_ok(need, workspace, ws_bytes)) return PARARNN_INVALID_ARG;
    const pararnn_norm_shape &s = *shape;
    if (!x || !stats || !dy || !dx || !aligned(x, 16) || !aligned(dy, 16) || !aligned(dx, 16) || !aligned(stats, 16) ||
        !aligned(weight, 16) || !aligned(bias, 16) || !aligned(gate, 16) || !aligned(dgate, 16) ||
        !aligned(dweight, 16) || !aligned(dbias, 16) || !aligned(lengths, 4))
        return PARARNN_INVALID_ARG;
    if ((gate == nullptr) != (dgate == nullptr)) return PARARNN_INVALID_ARG;
    const size_t n = static_cast<size_t>(s.N) * s.S * s.C, par = s.C * sizeof(float);
    const Extent out[] = {{dx, n * esize(s.x_dtype)}, {dgate, n * esize(s.x_dtype)}, {dweight, par}, {dbias, par},
                          {workspace, need == kNone ? 0 : need}};
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
