"""The selective state space block as it is used: its operators one after the other, a prompt against the same tokens one by
one, its gradients against differences, and calls next to one another.  Guard bands: every operand, output and workspace
between bands of 0xFF bytes, outputs starting as NaN and the workspace as 0xFF; the results are those of the same call on
ordinary allocations, bit for bit."""
import pytest
import torch

import newton_solve_nonlinear_b200 as fw
from newton_solve_nonlinear_b200 import binding
from tests.test_gpu_guard_bands import Guarded
from tests.test_gpu_layers_guard_bands import _done, _inputs, _stream, _ws

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


class Block:
    """norm -> projection to x and gate -> convolution -> projections to dt, b, c -> scan -> projection, in fp32."""

    def __init__(self, C=24, D=32, N=8, W=4, R=4, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s, std=1.0: std * torch.randn(*s, device="cuda", generator=g)
        self.C, self.D, self.N, self.W, self.R = C, D, N, W, R
        self.p = dict(norm=1 + 0.1 * n(C), w_in=n(C, 2 * D, std=C ** -0.5), conv=n(D, W, std=W ** -0.5), conv_b=0.1 * n(D),
                      w_x=n(D, R + 2 * N, std=D ** -0.5), w_dt=n(R, D, std=R ** -0.5), dt_b=n(D) - 2.0,
                      a=-torch.exp(0.5 * n(D, N)), skip=n(D), w_out=n(D, C, std=D ** -0.5))

    def start(self, B):
        return (torch.zeros(B, self.W - 1, self.D, device="cuda"), torch.zeros(B, self.D, self.N, device="cuda"))

    def forward(self, x, res, state, lengths=None):
        p, D, N, R = self.p, self.D, self.N, self.R
        B, T = x.shape[:2]
        y, r, stats = fw.layer_norm(x, p["norm"], residual=res, rms=True, lengths=lengths)
        xz = y @ p["w_in"]
        u, conv = fw.causal_conv(xz[..., :D], p["conv"], p["conv_b"], state=state[0], lengths=lengths)
        dbc = u @ p["w_x"]
        dt = dbc[..., :R] @ p["w_dt"]
        b, c = dbc[..., R:R + N].unflatten(2, (1, N)), dbc[..., R + N:].unflatten(2, (1, N))
        o, h, kept = fw.selective_scan(u, dt, p["a"], b, c, skip=p["skip"], gate=xz[..., D:], dt_bias=p["dt_b"], h0=state[1],
                                       lengths=lengths, keep=True)
        return o @ p["w_out"], r, (conv, h), (y, r, stats, xz, u, dbc, dt, b, c, o, kept, state, lengths)

    def backward(self, x, do, dr, saved):
        p, D, N, R = self.p, self.D, self.N, self.R
        y, r, stats, xz, u, dbc, dt, b, c, o, kept, state, lengths = saved
        dy = do @ p["w_out"].T
        g = fw.selective_scan_backward(u, dt, p["a"], b, c, dy, skip=p["skip"], gate=xz[..., D:], dt_bias=p["dt_b"], h0=state[1],
                                       lengths=lengths, kept=kept)
        ddbc = torch.cat([g["ddt"] @ p["w_dt"].T, g["db"].flatten(2), g["dc"].flatten(2)], -1)
        du = g["dx"] + ddbc @ p["w_x"].T
        k = fw.causal_conv_backward(xz[..., :D], p["conv"], du, p["conv_b"], state=state[0], lengths=lengths)
        dxz = torch.cat([k["dx"], g["dgate"]], -1)
        m = fw.layer_norm_backward(r, stats, dxz @ p["w_in"].T, p["norm"], dr=dr, rms=True, lengths=lengths)
        flat = lambda v: v.flatten(0, 1)
        return dict(x=m["dx"], norm=m["dweight"], w_in=flat(y).T @ flat(dxz), conv=k["dweight"], conv_b=k["dbias"],
                    w_x=flat(u).T @ flat(ddbc), w_dt=flat(dbc[..., :R]).T @ flat(g["ddt"]), dt_b=g["ddt_bias"], a=g["da"],
                    skip=g["dskip"], w_out=flat(o).T @ flat(do))

    def token(self, x, res, conv, h, slots=None):
        p, D, N, R = self.p, self.D, self.N, self.R
        y, r, _ = fw.layer_norm(x, p["norm"], residual=res, rms=True)
        xz = y @ p["w_in"]
        u = fw.causal_conv_step(xz[:, :D], p["conv"], conv, p["conv_b"], slots=slots)
        dbc = u @ p["w_x"]
        o = fw.selective_scan_step(u, dbc[:, :R] @ p["w_dt"], p["a"], dbc[:, R:R + N].unflatten(1, (1, N)),
                                   dbc[:, R + N:].unflatten(1, (1, N)), h, skip=p["skip"], gate=xz[:, D:], dt_bias=p["dt_b"],
                                   slots=slots)
        return o @ p["w_out"], r


def _xr(B, T, C, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(B, T, C, device="cuda", generator=g) for _ in range(2))


def test_a_prompt_and_its_tokens_one_by_one():
    """A padded batch as a prompt, then further tokens from a pool of states, against the whole as one prompt.  The
    projections are library products in fp32 (off by up to 2^-11 of a product's factors if run as TF32, which is off here)."""
    torch.backends.cuda.matmul.allow_tf32 = False
    blk, (B, T) = Block(), (3, 21)
    x, res = _xr(B, T, blk.C)
    lengths = [7, 1, 14]
    whole, r_whole, _, _ = blk.forward(x, res, blk.start(B))
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    y, r, (conv, h), _ = blk.forward(x, res, blk.start(B), ln)
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    convs, hs = torch.empty_like(conv), torch.empty_like(h)
    convs[slots.long()], hs[slots.long()] = conv, h
    for i, n in enumerate(lengths):
        torch.testing.assert_close(y[i, :n], whole[i, :n], rtol=2e-4, atol=2e-4)
    for step in range(7):
        at = torch.tensor([n + step for n in lengths], device="cuda")
        row = torch.arange(B, device="cuda")
        out, stream = blk.token(x[row, at], res[row, at], convs, hs, slots)
        torch.testing.assert_close(out, whole[row, at], rtol=2e-4, atol=2e-4)
        torch.testing.assert_close(stream, r_whole[row, at], rtol=1e-6, atol=1e-6)


@pytest.mark.parametrize("lengths", [None, [9, 0, 4]])
def test_gradients_against_differences(lengths):
    """Central differences along a random direction of each parameter: the loss in fp32 is off by 1e-6 of its terms, so a
    step of 1e-2 leaves 1e-3 of the slope next to the cubic term."""
    torch.backends.cuda.matmul.allow_tf32 = False
    blk, (B, T) = Block(C=12, D=16, N=4), (3, 9)
    x, res = _xr(B, T, blk.C, seed=2)
    do, dr = _xr(B, T, blk.C, seed=3)
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if ln is not None:
        on = (torch.arange(T, device="cuda")[None] < ln[:, None])[..., None]
        do, dr = do * on, dr * on

    def loss():
        y, r, _, _ = blk.forward(x, res, blk.start(B), ln)
        return float((y.double() * do).sum() + (r.double() * dr).sum())

    y, r, _, saved = blk.forward(x, res, blk.start(B), ln)
    grads = blk.backward(x, do, dr, saved)
    for name, g in grads.items():
        t = x if name == "x" else blk.p[name]
        step = torch.randn(t.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
        step *= 1e-2 / step.norm() * min(1.0, float(t.norm()))
        keep = t.clone()
        t.copy_(keep + step)
        up = loss()
        t.copy_(keep - step)
        down = loss()
        t.copy_(keep)
        want = float((g.double() * step).sum())
        size = float((g.double() * step).norm()) + abs(want)
        assert abs((up - down) / 2 - want) <= 2e-2 * size + 2e-4, name


def test_two_graphs_side_by_side():
    """Each call has its own workspace: two captured blocks replayed on two streams at once give what they give alone.  (Each
    is captured on a stream of its own: torch keeps the library products' workspace by stream.)"""
    blks = [Block(seed=s, D=64) for s in (0, 7)]
    xs = [tuple(_xr(2, 300, 24, seed=10 + i)) for i in range(2)]
    graphs, outs = [], []
    for blk, (x, res) in zip(blks, xs):
        run = lambda blk=blk, x=x, res=res: (lambda y, r, st, saved: (y, r, *st, *blk.backward(x, y, r, saved).values()))(
            *blk.forward(x, res, blk.start(2)))
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            outs.append(run())
        graphs.append(g)
    want = []
    for g, o in zip(graphs, outs):
        g.replay()
        torch.cuda.synchronize()
        want.append([t.clone() for t in o])
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for u, v in zip(o, w):
            assert torch.equal(u, v)


def test_a_stream_of_another_device_than_the_tensors_is_refused():
    x = torch.zeros(1, 2, 4, device="cuda")

    class Other:
        device = torch.device("cuda", 7)

    for call in (lambda s: fw.selective_scan(x, x, torch.zeros(4, 2, device="cuda"), x[..., :2, None].transpose(2, 3), x[..., :2, None].transpose(2, 3), stream=s),
                 lambda s: fw.causal_conv(x, torch.zeros(4, 2, device="cuda"), stream=s), lambda s: fw.layer_norm(x, stream=s)):
        with pytest.raises(ValueError, match="stream"):
            call(Other())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("B,T,G,per,N", [(1, 1, 1, 1, 1), (2, 33, 2, 7, 5), (2, 70, 1, 64, 16), (1, 500, 1, 24, 16), (3, 65, 1, 130, 33),
                                         (1, 17, 3, 10, 64), (2, 40, 1, 20, 8)])
def test_guard_bands_scan(B, T, G, per, N, ragged, dtype):
    L, D = binding.lib(), G * per
    st = (B, D, N)
    x = _inputs(x=((B, T, D), dtype), dt=((B, T, D), dtype), b=((B, T, G, N), dtype), c=((B, T, G, N), dtype), gate=((B, T, D), dtype),
                dy=((B, T, D), dtype), a=((D, N), F32), skip=((D,), F32), bias=((D,), F32), h0=(st, F32), dh=(st, F32))
    x["a"].t.copy_(-x["a"].t.abs())
    ln = Guarded((B,), torch.int32, init=torch.tensor([max(T - 3 * b, 0) for b in range(B)], device="cuda")) if ragged else None
    lens, t = None if ln is None else ln.t, {k: g.t for k, g in x.items()}
    ops = binding._scan_operands(t["x"], t["dt"], t["a"], t["b"], t["c"], t["skip"], t["gate"], t["bias"], True)
    p = lambda g: None if g is None else g.t.data_ptr()
    y, h, kept = Guarded((B, T, D), dtype), Guarded(st, F32), Guarded((B, (T + 7) // 8, D, N), F32)
    ws = _ws(L.pararnn_selective_scan_workspace_size(ops[0]))
    assert L.pararnn_selective_scan(*ops, p(x["h0"]), p(ln), p(y), p(h), p(kept), p(ws), ws.n, _stream()) == 0
    q = {k: g.t.clone() for k, g in x.items()}
    a, kw = (q["x"], q["dt"], q["a"], q["b"], q["c"]), dict(skip=q["skip"], gate=q["gate"], dt_bias=q["bias"], h0=q["h0"], lengths=lens)
    wy, wh, wk = fw.selective_scan(*a, keep=True, **kw)
    _done(dict(y=(y, wy), h=(h, wh)), [ws, *x.values()])
    assert kept.bands_intact()
    for i in range(B):
        n = ((T if lens is None else int(lens[i])) + 7) // 8
        assert torch.equal(kept.t[i, :n], wk[i, :n])

    rows, shared = (B, T, D), (B, T, G, N)
    for given in (True, False):
        g = dict(dx=Guarded(rows, dtype), ddt=Guarded(rows, dtype), da=Guarded((D, N), F32), db=Guarded(shared, dtype),
                 dc=Guarded(shared, dtype), dskip=Guarded((D,), F32), dgate=Guarded(rows, dtype), ddt_bias=Guarded((D,), F32),
                 dh0=Guarded(st, F32))
        ws = _ws(L.pararnn_selective_scan_backward_workspace_size(ops[0], int(given)))
        assert L.pararnn_selective_scan_backward(*ops, binding._plain_rows(t["dy"], "dy", t["x"], rows), p(x["h0"]), p(x["dh"]), p(ln),
                                                 p(kept) if given else None, *(p(v) for v in g.values()), p(ws), ws.n, _stream()) == 0
        want = fw.selective_scan_backward(*a, q["dy"], dh=q["dh"], kept=wk if given else None, **kw)
        _done({n: (g[n], want[n]) for n in g}, [ws, *x.values()])

    one = {k: Guarded((B, *g.t.shape[2:]), dtype, init=g.t[:, 0]) for k, g in x.items() if k in ("x", "dt", "b", "c", "gate")}
    u = {k: g.t for k, g in one.items()}
    ops1 = binding._scan_operands(u["x"], u["dt"], t["a"], u["b"], u["c"], t["skip"], u["gate"], t["bias"], True, 2)
    y1, out = Guarded((B, D), dtype), Guarded(st, F32)
    assert L.pararnn_selective_scan_step(*ops1, p(x["h0"]), None, B, p(y1), p(out), _stream()) == 0
    after = q["h0"].clone()
    w1 = fw.selective_scan_step(*(u[k].clone() for k in ("x", "dt")), q["a"], u["b"].clone(), u["c"].clone(), after, skip=q["skip"],
                                gate=u["gate"].clone(), dt_bias=q["bias"])
    _done(dict(y=(y1, w1), state=(out, after)), [*x.values(), *one.values()])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("B,T,D,W", [(1, 1, 1, 2), (2, 37, 5, 4), (3, 65, 24, 8), (2, 130, 66, 3), (1, 300, 128, 4)])
def test_guard_bands_conv(B, T, D, W, ragged, dtype):
    L, ends, rows = binding.lib(), (B, W - 1, D), (B, T, D)
    x = _inputs(x=(rows, dtype), dy=(rows, dtype), w=((D, W), F32), b=((D,), F32), state=(ends, dtype), dlast=(ends, dtype))
    ln = Guarded((B,), torch.int32, init=torch.tensor([max(T - 3 * b, 0) for b in range(B)], device="cuda")) if ragged else None
    lens, t = None if ln is None else ln.t, {k: g.t for k, g in x.items()}
    p = lambda g: None if g is None else g.t.data_ptr()
    s, r = binding._conv_shape(t["x"], t["w"], "silu"), lambda n: binding._plain_rows(t[n], n, t["x"], rows)
    y, last = Guarded(rows, dtype), Guarded(ends, dtype)
    assert L.pararnn_causal_conv(s, r("x"), p(x["w"]), p(x["b"]), p(x["state"]), p(ln), p(y), p(last), _stream()) == 0
    q = {k: g.t.clone() for k, g in x.items()}
    wy, wl = fw.causal_conv(q["x"], q["w"], q["b"], state=q["state"], lengths=lens)
    _done(dict(y=(y, wy), last=(last, wl)), x.values())
    g = dict(dx=Guarded(rows, dtype), dweight=Guarded((D, W), F32), dbias=Guarded((D,), F32), dstate=Guarded(ends, dtype))
    ws = _ws(L.pararnn_causal_conv_backward_workspace_size(s))
    assert L.pararnn_causal_conv_backward(s, r("x"), p(x["w"]), p(x["b"]), r("dy"), p(x["state"]), p(x["dlast"]), p(ln),
                                          *(p(v) for v in g.values()), p(ws), ws.n, _stream()) == 0
    want = fw.causal_conv_backward(q["x"], q["w"], q["dy"], q["b"], state=q["state"], dlast=q["dlast"], lengths=lens)
    _done({n: (g[n], want[n]) for n in g}, [ws, *x.values()])
    one = Guarded((B, D), dtype, init=t["x"][:, 0])
    y1, out = Guarded((B, D), dtype), Guarded(ends, dtype)
    s1 = binding._conv_shape(one.t, t["w"], "silu", 2)
    assert L.pararnn_causal_conv_step(s1, binding._plain_rows(one.t, "x", one.t, (B, D)), p(x["w"]), p(x["b"]), p(x["state"]), None, B,
                                      p(y1), p(out), _stream()) == 0
    after = q["state"].clone()
    w1 = fw.causal_conv_step(one.t.clone(), q["w"], after, q["b"])
    _done(dict(y=(y1, w1), state=(out, after)), [one, *x.values()])


@pytest.mark.parametrize("x_t,r_t,y_t", [(F32, F32, F32), (BF16, F32, BF16), (BF16, BF16, BF16)])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("N,S,C", [(1, 1, 1), (2, 3, 7), (3, 5, 132), (2, 4, 516), (1, 2, 1027), (1, 3, 2052), (2, 2, 8200), (1, 2, 33001)])
def test_guard_bands_norm(N, S, C, ragged, x_t, r_t, y_t):
    L, rows = binding.lib(), (N, S, C)
    x = _inputs(x=(rows, x_t), res=(rows, r_t), dy=(rows, y_t), dr=(rows, r_t), w=((C,), F32), b=((C,), F32))
    ln = Guarded((N,), torch.int32, init=torch.tensor([max(S - b, 0) for b in range(N)], device="cuda")) if ragged else None
    lens, t = None if ln is None else ln.t, {k: g.t for k, g in x.items()}
    p = lambda g: None if g is None else g.t.data_ptr()
    s = binding._stream_shape(t["x"], False, 1e-5, x_t, r_t, y_t)
    y, r, stats = Guarded(rows, y_t), Guarded(rows, r_t), Guarded((N, S, 2), F32)
    assert L.pararnn_layer_norm(s, p(x["x"]), p(x["res"]), p(x["w"]), p(x["b"]), p(ln), p(y), p(r), p(stats), _stream()) == 0
    q = {k: g.t.clone() for k, g in x.items()}
    wy, wr, ws_ = fw.layer_norm(q["x"], q["w"], q["b"], residual=q["res"], lengths=lens, out_dtype=y_t)
    _done(dict(y=(y, wy), r=(r, wr), stats=(stats, ws_)), x.values())
    g = dict(dr=Guarded(rows, r_t), dx=Guarded(rows, x_t) if x_t != r_t else None, dweight=Guarded((C,), F32), dbias=Guarded((C,), F32))
    ws = _ws(L.pararnn_layer_norm_backward_workspace_size(s))
    assert L.pararnn_layer_norm_backward(s, p(r), p(stats), p(x["dy"]), p(x["w"]), p(x["dr"]), p(ln), *(p(v) for v in g.values()),
                                         p(ws), ws.n, _stream()) == 0
    want = fw.layer_norm_backward(wr, ws_, q["dy"], q["w"], q["b"], dr=q["dr"], lengths=lens, dx_dtype=x_t)
    _done({n: (v, want[n]) for n, v in g.items() if v is not None}, [ws, *x.values()])
