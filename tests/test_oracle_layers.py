"""The fp64 oracles of linear attention and group norm: their gradients against central differences, and the
recurrence against the closed sum.  CPU only."""
import numpy as np
import pytest

from oracle import group_norm as gn
from oracle import linear_attention as la


def _diff(f, x, at, h=1e-5):
    x[at] += h
    up = f()
    x[at] -= 2 * h
    down = f()
    x[at] += h
    return (up - down) / (2 * h)


@pytest.mark.parametrize("H,Hkv,lengths", [(2, 2, None), (4, 2, [5, 0, 7])])
def test_linear_attention_gradients_against_differences(H, Hkv, lengths):
    r = np.random.default_rng(1)
    B, T, dk, dv = 3, 7, 3, 4
    q, k, v = r.normal(size=(B, T, H, dk)), r.normal(size=(B, T, Hkv, dk)), r.normal(size=(B, T, Hkv, dv))
    s0, ds, do = (r.normal(size=s) for s in ((B, H, dk, dv), (B, H, dk, dv), (B, T, H, dv)))
    ld = -np.linspace(0.0, 1.5, H)

    def loss():
        o, s = la.forward(q, k, v, ld, s0, lengths, 0.7)
        return float((o * do).sum() + (s * ds).sum())

    grads = la.backward(q, k, v, ld, do, s0, ds, lengths, 0.7)
    for x, g in zip((q, k, v, s0), grads):
        for at in [tuple(r.integers(0, n) for n in x.shape) for _ in range(12)]:
            assert abs(_diff(loss, x, at) - g[at]) <= 1e-7 * (1 + abs(g[at]))


def test_linear_attention_is_the_decayed_sum():
    r = np.random.default_rng(2)
    T, dk, dv = 9, 4, 5
    q, k, v = r.normal(size=(1, T, 1, dk)), r.normal(size=(1, T, 1, dk)), r.normal(size=(1, T, 1, dv))
    o, _ = la.forward(q, k, v, [-0.3], None, None, 0.5)
    w = np.tril(np.exp(-0.3 * (np.arange(T)[:, None] - np.arange(T)[None])))
    assert np.allclose(o[0, :, 0], 0.5 * (w * (q[0, :, 0] @ k[0, :, 0].T)) @ v[0, :, 0], atol=1e-12)


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
def test_group_norm_gradients_against_differences(kind, gated):
    r = np.random.default_rng(3)
    N, S, G, C = 3, 4, 2, 6
    x, dy, gate = (r.normal(size=(N, S, C)) for _ in range(3))
    w, b = r.normal(size=C), r.normal(size=C)
    gate = gate if gated else None
    lengths = [4, 0, 3]

    def loss():
        return float((gn.forward(x, G, w, b, gate, kind, 1e-5, lengths)[0] * dy).sum())

    grads = gn.backward(x, dy, G, w, b, gate, kind, 1e-5, lengths)
    for arr, g in zip((x, w, b, gate), grads):
        if arr is None:
            continue
        for at in [tuple(r.integers(0, n) for n in arr.shape) for _ in range(10)]:
            assert abs(_diff(loss, arr, at) - g[at]) <= 1e-6 * (1 + abs(g[at]))
