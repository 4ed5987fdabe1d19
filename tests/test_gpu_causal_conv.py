"""The short causal convolution on the GPU against fp64 and its running error bounds (oracle/causal_conv.py): elementwise
what fp32 may be off, and for results in bf16 half a step of 2^-8 of the value on top.  The last inputs are copies."""
import numpy as np
import pytest
import torch

import newton_solve_nonlinear_b200 as fw
from oracle import causal_conv as oracle
from tests.test_gpu_selective_scan import BF16, F32, _close, _np

pytestmark = pytest.mark.gpu


def _make(B, T, D, W, dtype, seed=0, full=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, dt=dtype: torch.randn(*s, device="cuda", generator=g).to(dt)
    p = dict(x=n(B, T, D), weight=n(D, W, dt=F32), bias=n(D, dt=F32) if full else None)
    return p, n(B, W - 1, D) if full else None, n


def _run(p, state, n, act, lengths=None, full=True):
    y, last = fw.causal_conv(**p, act=act, state=state, lengths=lengths)
    ln = None if lengths is None else lengths.tolist()
    q = {k: _np(v) for k, v in p.items()}
    want = oracle.forward(q["x"], q["weight"], q["bias"], act, _np(state), ln)
    _close(y, want["y"], "y")
    assert np.array_equal(_np(last), want["last"][0])
    dy, dlast = n(*y.shape), n(*last.shape) if full else None
    if ln is not None:
        for b, L in enumerate(ln):
            dy[b, max(L, 0):] = float("nan")
    g = fw.causal_conv_backward(p["x"], p["weight"], dy, p["bias"], act=act, state=state, dlast=dlast, lengths=lengths)
    for k, v in oracle.backward(q["x"], q["weight"], _np(dy), q["bias"], act, _np(state), _np(dlast), ln).items():
        _close(g[k], v, k)
    return y, last, g


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("B,T,D,W", [(1, 1, 1, 2), (2, 1, 8, 4), (1, 2, 5, 4), (3, 3, 4, 8), (2, 7, 12, 5), (1, 8, 33, 3), (2, 31, 16, 6),
                                     (1, 32, 130, 4), (2, 33, 64, 7), (1, 40, 257, 2), (3, 65, 24, 4), (2, 300, 40, 8), (1, 1000, 3, 4)])
def test_sizes(B, T, D, W, act, dtype):
    p, state, n = _make(B, T, D, W, dtype)
    _run(p, state, n, act)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_without_options(dtype):
    p, state, n = _make(2, 50, 20, 4, dtype, full=False)
    _run(p, state, n, "silu", full=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [16, 15])
@pytest.mark.parametrize("W,T,lengths", [(4, 100, [100, 0, 1, 2, 64]), (8, 70, [-3, 71, 3, 1 << 30, 33]), (3, 2, [2, 1, 0, 0, 1])])
def test_padded_batch(W, T, lengths, D, dtype):
    p, state, n = _make(5, T, D, W, dtype, seed=1)
    for b, L in enumerate(lengths):
        p["x"][b, min(max(L, 0), T):] = float("nan")
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    raw = fw.causal_conv(**p, state=state, lengths=ln)
    y, last, g = _run(p, state, n, "silu", ln.clamp(0, T))
    assert torch.equal(raw[0], y) and torch.equal(raw[1], last)
    for b, L in enumerate(lengths):
        L = min(max(L, 0), T)
        assert not y[b, L:].any() and not g["dx"][b, L:].any()
        if L == 0:
            assert torch.equal(last[b], state[b])


def test_a_token_that_is_not_finite_reaches_its_window_alone():
    for W in (3, 5, 8):
        p, state, _ = _make(1, 40, 8, W, F32, seed=2)
        p["x"][0, 10] = float("nan")
        y, _ = fw.causal_conv(**p, state=state)
        bad = torch.isnan(y[0]).any(1)
        assert bad.nonzero().flatten().tolist() == list(range(10, 10 + W))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("off", [0, 1])
def test_views(dtype, off):
    p, state, n = _make(2, 45, 24, 4, dtype, seed=3)
    wide = torch.empty(2, 45, 60, device="cuda", dtype=dtype)
    wide[..., off:off + 24] = p["x"]
    x = wide[..., off:off + 24]
    for u, v in zip(fw.causal_conv(x, p["weight"], p["bias"], state=state), fw.causal_conv(**p, state=state)):
        assert torch.equal(u, v)
    dy = n(1, 1, 24).expand(2, 45, 24)
    got = fw.causal_conv_backward(x, p["weight"], dy, p["bias"], state=state)
    want = fw.causal_conv_backward(p["x"], p["weight"], dy.contiguous(), p["bias"], state=state)
    for k in want:
        assert torch.equal(got[k], want[k]) if k != "dweight" and k != "dbias" else torch.allclose(got[k], want[k], rtol=1e-5, atol=1e-4)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,D,W,act", [(1, 1, 2, "silu"), (5, 24, 4, "silu"), (3, 33, 8, "none"), (2, 700, 3, "silu")])
def test_step_is_the_convolution_token_by_token(B, D, W, act, dtype):
    p, state, _ = _make(B, 12, D, W, dtype, seed=4)
    y, last = fw.causal_conv(**p, act=act, state=state)
    pool = torch.full((B + 3, W - 1, D), 7.0, device="cuda", dtype=dtype)
    slots = torch.randperm(B + 3, device="cuda")[:B].to(torch.int32)
    pool[slots.long()] = state
    for t in range(12):
        after = torch.full_like(pool, 3.0)
        out = fw.causal_conv_step(p["x"][:, t], p["weight"], pool, p["bias"], act=act, slots=slots, out_state=after)
        again = fw.causal_conv_step(p["x"][:, t], p["weight"], pool, p["bias"], act=act, slots=slots)
        assert torch.equal(out, again) and torch.equal(after[slots.long()], pool[slots.long()])
        q = {k: _np(v) for k, v in p.items()}
        want = oracle.forward(q["x"], q["weight"], q["bias"], act, _np(state))["y"]
        _close(out, (want[0][:, t], want[1][:, t]), f"y {t}")
    assert torch.equal(pool[slots.long()], last)
    rest = torch.ones(B + 3, dtype=torch.bool, device="cuda")
    rest[slots.long()] = False
    assert (pool[rest] == 7.0).all() and (after[rest] == 3.0).all()


@pytest.mark.parametrize("in_place", [True, False])
def test_step_slots_that_repeat_or_have_no_state(in_place):
    p, _, n = _make(6, 1, 40, 4, F32, seed=5)
    x, pool, ys = p["x"][:, 0], n(3, 3, 40), []
    want = pool.clone()
    for b, s in enumerate([1, -1, 1, 3, 0, 1]):
        if 0 <= s < 3:
            one = want[s:s + 1].clone()
            ys.append(fw.causal_conv_step(x[b:b + 1], p["weight"], one, p["bias"]))
            want[s] = one[0]
        else:
            ys.append(torch.zeros(1, 40, device="cuda"))
    slots = torch.tensor([1, -1, 1, 3, 0, 1], dtype=torch.int32, device="cuda")
    out = pool if in_place else pool.clone()
    y = fw.causal_conv_step(x, p["weight"], pool, p["bias"], slots=slots, out_state=out)
    assert torch.equal(y, torch.cat(ys)) and torch.equal(out, want)


def test_repeats_bit_for_bit_and_in_a_graph():
    p, state, n = _make(3, 500, 96, 4, BF16, seed=6)
    dy = n(3, 500, 96)
    run = lambda **k: (*fw.causal_conv(**p, state=state),
                       *fw.causal_conv_backward(p["x"], p["weight"], dy, p["bias"], state=state, **k).values())
    first = run()
    for fill in (0x00, 0xFF):
        for u, v in zip(run(workspace=torch.full((1 << 22,), fill, dtype=torch.uint8, device="cuda")), first):
            assert torch.equal(u, v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    p["x"].copy_(n(3, 500, 96)), dy.copy_(n(3, 500, 96))
    graph.replay()
    torch.cuda.synchronize()
    for u, v in zip(out, run()):
        assert torch.equal(u, v)


def test_refusals():
    p, state, n = _make(2, 10, 8, 4, F32, seed=7)
    for kw in (dict(state=state[:, :2]), dict(state=state.bfloat16()), dict(lengths=torch.zeros(2, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            fw.causal_conv(**p, **kw)
    with pytest.raises(ValueError):
        fw.causal_conv(p["x"].transpose(1, 2), torch.randn(10, 4, device="cuda"))
    with pytest.raises(RuntimeError):  # the last inputs over the state that first tokens still read
        fw.causal_conv(**p, state=state, out=(torch.empty_like(p["x"]), state))
