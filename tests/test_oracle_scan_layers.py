"""The fp64 oracles of the selective scan, the causal convolution and the stream's norm: their gradients against central
differences, and their bounds against an fp32 evaluation.  CPU only."""
import numpy as np
import pytest

from oracle import bounds, causal_conv, layer_norm
from oracle.selective_scan import Scan


def _diff(f, x, at, h=1e-5):
    x[at] += h
    up = f()
    x[at] -= 2 * h
    down = f()
    x[at] += h
    return (up - down) / (2 * h)


def _check(loss, pairs, r, n=8):
    for x, g in pairs:
        if x is None:
            assert g is None
            continue
        for at in [tuple(r.integers(0, k) for k in x.shape) for _ in range(n)]:
            assert abs(_diff(loss, x, at) - g[0][at]) <= 1e-6 * (1 + abs(g[0][at]))


@pytest.mark.parametrize("soft", [True, False])
@pytest.mark.parametrize("full", [True, False])
@pytest.mark.parametrize("lengths", [None, [5, 0, 7]])
def test_scan_gradients_against_differences(full, soft, lengths):
    r = np.random.default_rng(1)
    B, T, G, D, N = 3, 7, 2, 4, 3
    n = lambda *s: r.normal(size=s)
    x, dt, b, c, a = n(B, T, D), n(B, T, D), n(B, T, G, N), n(B, T, G, N), -np.exp(n(D, N))
    dt = dt if soft else np.abs(dt)
    opt = dict(skip=n(D), gate=n(B, T, D), dt_bias=n(D) if soft else np.abs(n(D)), h0=n(B, D, N)) if full else {}
    dy, dh = n(B, T, D), n(B, D, N)

    def loss():
        out = Scan(x, dt, a, b, c, use_softplus=soft, lengths=lengths, **opt).forward()
        return float((out["y"][0] * dy).sum() + (out["h"][0] * dh).sum())

    g = Scan(x, dt, a, b, c, use_softplus=soft, lengths=lengths, **opt).backward(dy, dh)
    _check(loss, [(x, g["dx"]), (dt, g["ddt"]), (a, g["da"]), (b, g["db"]), (c, g["dc"]), (opt.get("skip"), g["dskip"]),
                  (opt.get("gate"), g["dgate"]), (opt.get("dt_bias"), g["ddt_bias"]), (opt.get("h0"), g["dh0"])], r)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("W,T", [(2, 5), (4, 6), (8, 3)])
@pytest.mark.parametrize("lengths", [None, [0, 2]])
def test_conv_gradients_against_differences(act, W, T, lengths):
    r = np.random.default_rng(2)
    B, D = 2, 3
    n = lambda *s: r.normal(size=s)
    x, w, bias, state, dy, dlast = n(B, T, D), n(D, W), n(D), n(B, W - 1, D), n(B, T, D), n(B, W - 1, D)

    def loss():
        out = causal_conv.forward(x, w, bias, act, state, lengths)
        return float((out["y"][0] * dy).sum() + (out["last"][0] * dlast).sum())

    g = causal_conv.backward(x, w, dy, bias, act, state, dlast, lengths)
    _check(loss, [(x, g["dx"]), (w, g["dweight"]), (bias, g["dbias"]), (state, g["dstate"])], r)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("lengths", [None, [4, 0, 2]])
def test_norm_gradients_against_differences(rms, lengths):
    r = np.random.default_rng(3)
    x, res, dy, dr = (r.normal(size=(3, 4, 6)) for _ in range(4))
    w, b = r.normal(size=6), r.normal(size=6)

    def loss():
        out = layer_norm.forward(x, res, w, b, rms, 1e-5, lengths)
        return float((out["y"][0] * dy).sum() + (out["r"][0] * dr).sum())

    out = layer_norm.forward(x, res, w, b, rms, 1e-5, lengths)
    g = layer_norm.backward(out["r"][0], out["stats"][0], dy, w, dr, rms, lengths)
    _check(loss, [(x, g["dr"]), (res, g["dr"]), (w, g["dweight"]), (b, g["dbias"])], r)


def test_bounds_hold_for_an_fp32_evaluation():
    """The same recurrence in numpy's fp32 stays within the bounds, and uses a fair part of them."""
    r = np.random.default_rng(4)
    B, T, G, D, N = 2, 60, 1, 5, 4
    f = lambda *s: r.normal(size=s).astype(np.float32)
    x, dt, b, c, a = f(B, T, D), f(B, T, D), f(B, T, G, N), f(B, T, G, N), -np.exp(f(D, N))
    s = np.log1p(np.exp(dt))
    h, y = np.zeros((B, D, N), np.float32), np.zeros((B, T, D), np.float32)
    for t in range(T):
        e = np.expm1(s[:, t, :, None] * a)
        h = h + e * h + (s[:, t] * x[:, t])[..., None] * b[:, t]
        y[:, t] = (c[:, t] * h).sum(-1)
    o = Scan(*(v.astype(np.float64) for v in (x, dt, a, b, c))).forward()
    part = np.abs(y - o["y"][0]) / o["y"][1]
    assert 1e-3 < part.max() <= 1.0
    assert (np.abs(h - o["h"][0]) <= o["h"][1]).all()


def test_silu_slope_bound():
    z = np.linspace(-30, 30, 4001).astype(np.float32)
    one = np.float32(1)
    s = one / (one + np.exp(-z))
    got = s * (one + z * (one - s))
    z = z.astype(np.float64)
    assert (np.abs(got - bounds.silu_slope(z)) <= bounds.silu_slope_bound(z).e + 1e-30).all()
