"""The selective scan on the GPU against the fp64 recurrence and its running error bounds (oracle/selective_scan.py).

Tolerances are elementwise: what an fp32 evaluation of the recurrence may be off (bounds.Bound: half a step, 2^-24, for each
product and sum, and the stated errors of the step, the decay and the gate, carried through the recurrence), and for
results in bf16 their rounding, half a step of 2^-8 of the value, on top."""
import numpy as np
import pytest
import torch

import newton_solve_nonlinear_b200 as fw
from oracle.selective_scan import Scan

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _make(B, T, G, per, N, dtype, seed=0, full=True, soft=True, rate=1.0, step=0.05):
    """Operands of a call; steps around `step`, rates around `rate` .. `rate` N."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, dt=dtype: torch.randn(*s, device="cuda", generator=g).to(dt)
    D = G * per
    a = -rate * torch.arange(1, N + 1, device="cuda") * torch.exp(0.3 * n(D, N, dt=F32))
    p = dict(x=n(B, T, D), dt=n(B, T, D), a=a, b=n(B, T, G, N), c=n(B, T, G, N))
    raw = float(np.log(np.expm1(step)))
    o = dict(softplus=soft)
    if full:
        o.update(skip=n(D, dt=F32), gate=n(B, T, D), h0=n(B, D, N, dt=F32),
                 dt_bias=n(D, dt=F32) * 0.5 + raw if soft else None)
    elif soft:
        p["dt"] = (p["dt"].float() + raw).to(dtype)
    if not soft:
        p["dt"] = (step * torch.exp(p["dt"].float())).to(dtype)
    return p, o, n


def _oracle(p, o, lengths=None):
    q = {k: _np(v) for k, v in p.items()}
    r = {k: _np(v) if torch.is_tensor(v) else v for k, v in o.items() if k != "softplus"}
    return Scan(*(q[k] for k in ("x", "dt", "a", "b", "c")), use_softplus=o["softplus"], lengths=lengths, **r)


def _close(got, want, what):
    if want is None:
        assert got is None, what
        return
    value, bound = want
    g = _np(got)
    assert g.shape == value.shape and np.all(np.isfinite(g)), what
    tol = bound + 1e-30
    if got.dtype == BF16:
        tol = tol + 2.0 ** -8 * (np.abs(value) + bound)
    worst = float(np.max(np.abs(g - value) / tol)) if g.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times the tolerance"


def _forward(p, o, lengths=None, **kw):
    out = fw.selective_scan(*p.values(), lengths=lengths, **o, **kw)
    oracle = _oracle(p, o, None if lengths is None else lengths.tolist())
    want = oracle.forward()
    _close(out[0], want["y"], "y")
    _close(out[1], want["h"], "h")
    return out, oracle


def _both(p, o, n, lengths=None, dh=True):
    (y, h, kept), oracle = _forward(p, o, lengths, keep=True)
    B, T, D = p["x"].shape
    dy = n(B, T, D)
    dh = n(*h.shape, dt=F32) if dh else None
    if lengths is not None:
        for b, L in enumerate(lengths.tolist()):
            dy[b, max(L, 0):] = float("nan")
    g = fw.selective_scan_backward(*p.values(), dy, dh=dh, lengths=lengths, kept=kept, **o)
    for k, v in oracle.backward(_np(dy), _np(dh)).items():
        _close(g[k], v, k)
    again = fw.selective_scan_backward(*p.values(), dy, dh=dh, lengths=lengths, **o)  # without the kept states
    for k, v in g.items():
        assert (v is None and again[k] is None) or torch.equal(v, again[k]), k
    return g


SIZES = [
    # B, T, G, channels of a group, N
    (1, 1, 1, 1, 1), (2, 1, 2, 3, 16), (1, 2, 1, 5, 3), (3, 7, 1, 33, 4), (2, 8, 3, 7, 5), (2, 9, 1, 64, 16), (1, 15, 2, 65, 8),
    (1, 16, 1, 31, 9), (2, 17, 1, 130, 16), (1, 33, 1, 20, 17), (1, 40, 1, 17, 32), (2, 65, 2, 9, 33), (1, 100, 1, 12, 64),
    (1, 128, 1, 257, 2), (1, 129, 5, 3, 63), (2, 300, 1, 40, 16), (1, 1025, 1, 6, 16), (5, 257, 1, 4, 7),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", SIZES)
def test_forward(size, dtype):
    p, o, _ = _make(*size, dtype)
    _forward(p, o)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", SIZES)
def test_backward(size, dtype):
    p, o, n = _make(*size, dtype, seed=1)
    _both(p, o, n)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("full", [True, False])
@pytest.mark.parametrize("soft", [True, False])
def test_without_options(full, soft, dtype):
    p, o, n = _make(2, 75, 2, 20, 16, dtype, full=full, soft=soft, seed=2)
    _both(p, o, n, dh=full)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,lengths", [(200, [200, 0, 1, 129, 128]), (700, [0, 699, 64, 513, 7]), (70, [-3, 71, 69, 1 << 30, 33]),
                                       (9, [8, 9, 0, 0, 0])])
def test_padded_batch(T, lengths, dtype):
    p, o, n = _make(5, T, 2, 10, 12, dtype, seed=3)
    for b, L in enumerate(lengths):
        for t in (p["x"], p["dt"], p["b"], p["c"], o["gate"]):
            t[b, min(max(L, 0), T):] = float("nan") if b % 2 else float("inf")
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    y, h = fw.selective_scan(*p.values(), lengths=ln, **o)
    g = _both(p, o, n, ln.clamp(0, T))
    for b, L in enumerate(lengths):
        L = min(max(L, 0), T)
        assert not y[b, L:].any()
        for k in ("dx", "ddt", "dgate", "db", "dc"):
            assert not g[k][b, L:].any(), k
        if L == 0:
            assert torch.equal(h[b], o["h0"][b])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rate,step", [(1e-3, 0.002), (0.02, 0.01), (30.0, 0.5), (1.0, 5.0)])
def test_decays_from_slow_to_all(rate, step, dtype):
    """Memories of 5e5 tokens and states that a token replaces."""
    p, o, n = _make(1, 500, 1, 24, 16, dtype, rate=rate, step=step, seed=4)
    p["a"][0, :3] = torch.tensor([0.0, -1e-6, -1e4], device="cuda")
    _both(p, o, n)


def test_slow_decays_keep_their_rate():
    """8192 tokens of a memory of 1e6."""
    T, D = 8192, 32
    x = torch.ones(1, T, D, device="cuda")
    dt, a = torch.full((1, T, D), 1e-3, device="cuda"), torch.full((D, 1), -1e-3, device="cuda")
    b = torch.zeros(1, T, 1, 1, device="cuda")
    h0 = torch.ones(1, D, 1, device="cuda")
    _, h = fw.selective_scan(x, dt, a, b, b, softplus=False, h0=h0)
    # h stays in [1/2, 1], so each token's rounding of h + (exp(s a) - 1) h moves it by up to 2^-25; what else is off is
    # in exp(s a) - 1 = -1e-6, by parts of 1e-7 of it
    want = float(np.exp(-T * float(np.float32(1e-3)) ** 2))
    assert float((h - want).abs().max()) <= 8192 * 2.0 ** -25


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_views_of_one_projection(dtype):
    """x and gate, and dt, b and c, are slices of two tensors, at odd offsets; dy is expanded."""
    p, o, n = _make(2, 90, 2, 21, 9, dtype, seed=5)
    B, T, D = p["x"].shape
    xz = torch.empty(B, T, 2 * D + 1, device="cuda", dtype=dtype)
    rest = torch.empty(B, T, D + 4 * 9 + 3, device="cuda", dtype=dtype)
    xz[..., 1:1 + D], xz[..., 1 + D:] = p["x"], o["gate"]
    rest[..., 1:1 + D], rest[..., 2 + D:20 + D], rest[..., 20 + D:38 + D] = p["dt"], p["b"].flatten(2), p["c"].flatten(2)
    q = dict(x=xz[..., 1:1 + D], dt=rest[..., 1:1 + D], a=p["a"], b=rest[..., 2 + D:20 + D].unflatten(2, (2, 9)),
             c=rest[..., 20 + D:38 + D].unflatten(2, (2, 9)))
    oq = dict(o, gate=xz[..., 1 + D:])
    for u, v in zip(fw.selective_scan(*q.values(), keep=True, **oq), fw.selective_scan(*p.values(), keep=True, **o)):
        assert torch.equal(u, v)
    dy = n(1, 1, D).expand(B, T, D)
    got, want = (fw.selective_scan_backward(*k.values(), dy, **m) for k, m in ((q, oq), (p, o)))
    for k in want:
        assert torch.equal(got[k], want[k]), k
    # transposed in batch and time, and one sequence for all of the batch
    t = lambda v: v.transpose(0, 1).contiguous().transpose(0, 1)
    got = fw.selective_scan(*(t(v) if v.dim() > 2 else v for v in p.values()), **dict(o, gate=t(o["gate"])))
    assert torch.equal(got[0], fw.selective_scan(*p.values(), **o)[0])
    one = {k: v[:1].expand_as(v) if v.dim() > 2 else v for k, v in p.items()}
    y, _ = fw.selective_scan(*one.values(), softplus=o["softplus"], dt_bias=o["dt_bias"])
    assert torch.equal(y[0], y[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_few_channels_and_many_tokens(dtype):
    """Split into segments of time."""
    p, o, n = _make(1, 6000, 1, 3, 16, dtype, seed=6)
    _both(p, o, n)


def test_carried_state_over_parts():
    """A sequence in parts, each from the last one's state, and token by token, is the whole sequence."""
    p, o, _ = _make(2, 100, 1, 20, 16, F32, seed=7)
    y, h = fw.selective_scan(*p.values(), **o)
    state, at = o["h0"], 0
    for n in (1, 30, 8, 61):
        cut = lambda v: v[:, at:at + n]
        q = {k: cut(v) if v.dim() > 2 else v for k, v in p.items()}
        part, state = fw.selective_scan(*q.values(), **dict(o, h0=state, gate=cut(o["gate"])))
        assert torch.allclose(part, cut(y), rtol=1e-4, atol=1e-4)
        at += n
    oracle = _oracle(p, o)
    want = oracle.forward()
    _close(state, want["h"], "h")
    pool, ys = o["h0"].clone(), []
    for t in range(100):
        q = {k: v[:, t] if v.dim() > 2 else v for k, v in p.items()}
        ys.append(fw.selective_scan_step(*q.values(), pool, **{k: v[:, t] if k == "gate" else v for k, v in o.items() if k != "h0"}))
    _close(torch.stack(ys, 1), want["y"], "y")
    _close(pool, want["h"], "h")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,G,per,N", [(1, 1, 1, 1), (3, 1, 50, 16), (5, 2, 33, 5), (2, 1, 300, 64), (7, 3, 20, 8)])
def test_step(B, G, per, N, dtype):
    p, o, n = _make(B, 1, G, per, N, dtype, seed=8)
    want = _oracle(p, o).forward()
    q = {k: v[:, 0] if v.dim() > 2 else v for k, v in p.items()}
    m = {k: v[:, 0] if k == "gate" else v for k, v in o.items() if k != "h0"}
    D = G * per
    pool = n(B + 4, D, N, dt=F32)
    slots = torch.randperm(B + 4, device="cuda")[:B].to(torch.int32)
    pool[slots.long()] = o["h0"]
    before, after = pool.clone(), torch.full_like(pool, 7.0)
    y = fw.selective_scan_step(*q.values(), pool, slots=slots, out_state=after, **m)
    _close(y[:, None], want["y"], "y")
    _close(after[slots.long()], want["h"], "state")
    assert torch.equal(pool, before)
    rest = torch.ones(B + 4, dtype=torch.bool, device="cuda")
    rest[slots.long()] = False
    assert (after[rest] == 7.0).all()
    assert torch.equal(fw.selective_scan_step(*q.values(), pool, slots=slots, **m), y)  # in place
    assert torch.equal(pool[slots.long()], after[slots.long()]) and torch.equal(pool[rest], before[rest])
    direct = o["h0"].clone()
    assert torch.equal(fw.selective_scan_step(*q.values(), direct, **m), y)
    assert torch.equal(direct, pool[slots.long()])


@pytest.mark.parametrize("in_place", [True, False])
def test_step_slots_that_repeat_or_have_no_state(in_place):
    p, o, n = _make(6, 1, 1, 40, 16, F32, seed=9)
    q = {k: v[:, 0] if v.dim() > 2 else v for k, v in p.items()}
    m = {k: v[:, 0] if k == "gate" else v for k, v in o.items() if k != "h0"}
    pool = n(3, 40, 16, dt=F32)
    want, ys = pool.clone(), []
    for b, s in enumerate([1, -1, 1, 3, 0, 1]):
        if 0 <= s < 3:
            row = {k: v[b:b + 1] if k not in ("a",) else v for k, v in q.items()}
            one = want[s:s + 1].clone()
            ys.append(fw.selective_scan_step(*row.values(), one, **{k: v[b:b + 1] if k == "gate" else v for k, v in m.items()}))
            want[s] = one[0]
        else:
            ys.append(torch.zeros(1, 40, device="cuda"))
    slots = torch.tensor([1, -1, 1, 3, 0, 1], dtype=torch.int32, device="cuda")
    out = pool if in_place else pool.clone()
    y = fw.selective_scan_step(*q.values(), pool, slots=slots, out_state=out, **m)
    assert torch.equal(y, torch.cat(ys)) and torch.equal(out, want)


def test_state_in_place_and_given_outputs():
    p, o, _ = _make(2, 300, 1, 12, 16, F32, seed=10)
    y, h = fw.selective_scan(*p.values(), **o)
    state, out = o["h0"].clone(), torch.full_like(y, float("nan"))
    a = fw.selective_scan(*p.values(), **dict(o, h0=state), out=(out, state))
    assert a[0] is out and a[1] is state and torch.equal(out, y) and torch.equal(state, h)


def test_repeats_bit_for_bit_with_any_workspace():
    p, o, n = _make(2, 700, 2, 30, 16, BF16, seed=11)
    dy = n(*p["x"].shape)
    first = fw.selective_scan_backward(*p.values(), dy, **o)
    y = fw.selective_scan(*p.values(), **o)
    for fill in (0x00, 0xFF):
        ws = torch.full((1 << 24,), fill, dtype=torch.uint8, device="cuda")
        for u, v in zip(fw.selective_scan(*p.values(), **o, workspace=ws), y):
            assert torch.equal(u, v)
        for k, v in fw.selective_scan_backward(*p.values(), dy, **o, workspace=ws).items():
            assert torch.equal(v, first[k]), k


def test_graph_of_a_training_step():
    """Captured with a workspace of its own, replayed on other inputs."""
    p, o, n = _make(2, 260, 1, 24, 16, BF16, seed=12)
    dy = n(*p["x"].shape)

    def step():
        y, h, kept = fw.selective_scan(*p.values(), keep=True, **o)
        return dict(fw.selective_scan_backward(*p.values(), dy, kept=kept, **o), y=y, h=h)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t in (p["x"], p["b"], o["gate"], dy):
        t.copy_(n(*t.shape))
    graph.replay()
    torch.cuda.synchronize()
    for k, v in step().items():
        assert torch.equal(out[k], v), k


def test_on_a_stream_of_its_own():
    p, o, n = _make(2, 260, 1, 24, 16, F32, seed=13)
    want = fw.selective_scan(*p.values(), **o)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fw.selective_scan(*p.values(), **o, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for u, v in zip(got, want):
        assert torch.equal(u, v)


def test_refuses_to_drop_a_gradient_and_wrong_operands():
    p, o, n = _make(2, 10, 1, 8, 4, F32, seed=14)
    with pytest.raises(ValueError, match="no_grad"):
        fw.selective_scan(*{**p, "dt": p["dt"].clone().requires_grad_()}.values(), **o)
    with torch.no_grad():
        fw.selective_scan(*{**p, "dt": p["dt"].clone().requires_grad_()}.values(), **o)
    for k, v in (("dt", p["dt"][:, :5]), ("b", p["b"][..., :3]), ("c", p["c"].transpose(1, 2)), ("a", p["a"].T)):
        with pytest.raises(ValueError):
            fw.selective_scan(*{**p, k: v}.values(), **o)
    with pytest.raises(TypeError):
        fw.selective_scan(*{**p, "b": p["b"].bfloat16()}.values(), **o)
    for kw in (dict(h0=o["h0"][:1]), dict(skip=o["skip"].cpu()), dict(gate=o["gate"][..., :4])):
        with pytest.raises(ValueError):
            fw.selective_scan(*p.values(), **{**o, **kw})
    with pytest.raises(ValueError):
        fw.selective_scan_backward(*p.values(), n(2, 10, 8), **o, kept=n(2, 1, 8, 4, dt=F32))
