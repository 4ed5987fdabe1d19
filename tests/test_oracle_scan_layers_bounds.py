"""The selective scan's error bounds are those of fp32 for fast decays too: they follow exp(s a), however small it is, so that a
kernel whose fast decays had no digits left would not pass them.  CPU only."""
import numpy as np
import pytest

from oracle.bounds import U
from oracle.selective_scan import Scan


def _positive(T, rate, seed=0):
    """A step of 1, rates around `rate`, all else positive: no sum cancels."""
    r = np.random.default_rng(seed)
    B, D, N = 2, 3, 4
    u = lambda *s: r.uniform(0.5, 1.5, s)
    p = dict(x=10 ** r.uniform(-5, 4, (B, T, D)), dt=np.ones((B, T, D)), a=-rate * u(D, N), b=u(B, T, 1, N), c=u(B, T, 1, N))
    return p, 100 * u(B, D, N), u(B, T, D), u(B, D, N)


@pytest.mark.parametrize("rate", [3.0, 8.0, 16.0, 25.0])
@pytest.mark.parametrize("T", [1, 4, 30])
def test_bounds_of_fast_decays_are_relative(rate, T):
    """z off by (es + 2 U) |a|, |a| up to 38, and ex2 by 4 U, products and sums: 200 U of a value, twice that of a product of two,
    and n U for a sum of n."""
    p, h0, dy, dh = _positive(T, rate)
    scan = Scan(**p, use_softplus=False, h0=h0, joined=0)
    out = scan.forward()
    out.update(scan.backward(dy, dh))
    for k, steps in dict(h=200, y=200, dh0=200, da=400 + 2 * T, db=200, dc=200).items():
        value, bound = out[k]
        assert (bound <= steps * U * np.abs(value)).all(), (k, float((bound / np.abs(value)).max() / U))


@pytest.mark.parametrize("rate", [12.0, 16.0, 25.0])
def test_bounds_refuse_decays_as_a_difference_from_one(rate):
    """The same recurrence in fp32 with 1 + (exp(z) - 1) for exp(z) is outside of them, in the states and in da and dh0."""
    f = np.float32
    p, h0, dy, dh = _positive(6, rate, seed=1)
    p = {k: v.astype(f).astype(np.float64) for k, v in p.items()}
    h0, dy, dh = (v.astype(f).astype(np.float64) for v in (h0, dy, dh))
    scan = Scan(**p, use_softplus=False, h0=h0)
    want = scan.forward()
    want.update(scan.backward(dy, dh))
    for kept in (False, True):  # False: the difference from one; True: exp(z) itself
        w = np.exp(p["a"].astype(f)) if kept else None
        e = None if kept else np.expm1(p["a"].astype(f))
        hs = [h0.astype(f)]
        for t in range(6):
            ub = (p["x"][:, t, :, None].astype(f) * p["b"][:, t].astype(f))
            hs.append(w * hs[-1] + ub if kept else hs[-1] + ub + e * hs[-1])
        P, da = dh.astype(f), np.zeros_like(p["a"], dtype=f)
        for t in reversed(range(6)):
            g = P + dy[:, t, :, None].astype(f) * p["c"][:, t].astype(f)
            P = w * g if kept else g + e * g
            da = da + (P * hs[t]).sum(0)
        inside = {k: (np.abs(got - want[k][0]) <= want[k][1]).all() for k, got in dict(h=hs[-1], da=da, dh0=P).items()}
        assert all(v == kept for v in inside.values()), inside


def test_bounds_hold_for_an_fp32_evaluation_with_slow_and_fast_decays():
    """Rates from 1e-3 to 20, softplus and a gate, in numpy's fp32 with each decay in its own form."""
    f = np.float32
    r = np.random.default_rng(5)
    B, T, D, N = 2, 80, 6, 5
    n = lambda *s: r.normal(size=s).astype(f)
    x, dt, b, c = n(B, T, D), n(B, T, D), n(B, T, 1, N), n(B, T, 1, N)
    a = -np.exp(r.uniform(np.log(1e-3), np.log(20), (D, N))).astype(f)
    s = np.log1p(np.exp(dt))
    h, y = np.zeros((B, D, N), f), np.zeros((B, T, D), f)
    for t in range(T):
        z = s[:, t, :, None] * a
        slow = np.abs(z) < 0.0108
        h = np.where(slow, np.expm1(z), np.exp(z)) * h + ((s[:, t] * x[:, t])[..., None] * b[:, t] + np.where(slow, h, f(0)))
        y[:, t] = (c[:, t] * h).sum(-1)
    o = Scan(*(v.astype(np.float64) for v in (x, dt, a, b, c)), joined=0).forward()
    for got, (value, bound) in ((y, o["y"]), (h, o["h"])):
        part = np.abs(got - value) / bound
        assert 1e-3 < part.max() <= 1.0
