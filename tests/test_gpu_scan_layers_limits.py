"""The state space block's calls at the edges of what the header allows: operands of more than 2^31 elements, a group for
every channel, steps of zero from -inf, the most taps, states and tokens of odd counts."""
import pytest
import torch

import newton_solve_nonlinear_b200 as fw
from tests.test_gpu_selective_scan import BF16, F32, _both, _close, _make, _oracle

pytestmark = pytest.mark.gpu


def _rows(n, *shape, dtype=BF16):
    """n random rows repeated along the second axis: large operands without a large generator run."""
    x = torch.randn(1, n, *shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(dtype)
    return lambda T: x.repeat(1, T // n + 1, *[1] * len(shape))[:, :T]


def test_scan_of_more_than_2_31_elements():
    """The last tokens of 2^20 + 77 of 2048 channels against a call on them alone, from the state before them.  Both follow
    the same recurrence in fp32; they differ by the chunks' and segments' roundings, 1e-3 of the outputs' spread at most."""
    T, D, N, tail = (1 << 20) + 77, 2048, 4, 64
    x, dt = _rows(257, D)(T), _rows(61, D)(T)
    b, c = _rows(31, 1, N)(T), _rows(37, 1, N)(T)
    a = -torch.arange(1, N + 1, device="cuda", dtype=F32).repeat(D, 1)
    bias = torch.full((D,), -4.0, device="cuda")
    assert x.numel() > 2 ** 31
    y, h = fw.selective_scan(x, dt, a, b, c, dt_bias=bias)
    n = torch.tensor([T - tail], dtype=torch.int32, device="cuda")
    cut, before = fw.selective_scan(x, dt, a, b, c, dt_bias=bias, lengths=n)
    assert not cut[0, T - tail:].any() and torch.equal(cut[0, :1000], y[0, :1000])
    end = lambda v: v[:, T - tail:]
    ye, he = fw.selective_scan(end(x), end(dt), a, end(b), end(c), dt_bias=bias, h0=before)
    torch.testing.assert_close(he, h, rtol=1e-4, atol=1e-5)
    torch.testing.assert_close(ye.float(), end(y).float(), rtol=2 ** -7, atol=1e-3)


def test_conv_of_more_than_2_31_elements():
    T, D, tail = (1 << 20) + 77, 2048, 100
    x = _rows(257, D)(T)
    w = torch.randn(D, 4, device="cuda")
    y, last = fw.causal_conv(x, w)
    ye, le = fw.causal_conv(x[:, T - tail:], w, state=x[:, T - tail - 3:T - tail].contiguous())
    assert torch.equal(ye, y[:, T - tail:]) and torch.equal(le, last) and torch.equal(last, x[:, T - 3:])
    dy = y
    g = fw.causal_conv_backward(x, w, dy)
    e = fw.causal_conv_backward(x[:, T - tail:], w, dy[:, T - tail:], state=x[:, T - tail - 3:T - tail].contiguous())
    assert torch.equal(e["dx"], g["dx"][:, T - tail:])


def test_norm_of_more_than_2_31_elements():
    rows, C, tail = (1 << 20) + 77, 2048, 100
    x = _rows(257, C)(rows)[0]
    w = torch.randn(C, device="cuda")
    y, r, stats = fw.layer_norm(x, w, residual=x)
    ye, re, se = fw.layer_norm(x[rows - tail:].contiguous(), w, residual=x[rows - tail:].contiguous())
    assert torch.equal(ye, y[rows - tail:]) and torch.equal(re, r[rows - tail:]) and torch.equal(se, stats[rows - tail:])
    g = fw.layer_norm_backward(r, stats, y, w)
    e = fw.layer_norm_backward(re, se, ye, w)
    assert torch.equal(e["dr"], g["dr"][rows - tail:])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,G,per,N", [(2, 20, 37, 1, 16), (1, 9, 64, 2, 3), (1, 33, 1, 1, 64)])
def test_a_group_for_every_channel_or_two(B, T, G, per, N, dtype):
    p, o, n = _make(B, T, G, per, N, dtype, seed=21)
    _both(p, o, n)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_step_of_minus_infinity_leaves_the_state(dtype):
    """softplus(-inf) = 0: such a token adds nothing and decays nothing, as one of the type's lowest value."""
    p, o, _ = _make(2, 50, 1, 12, 8, dtype, seed=22)
    p["dt"][0, 10:30] = float("-inf")
    p["dt"][1, 5:] = torch.finfo(dtype).min
    y, h = fw.selective_scan(*p.values(), **o)
    assert torch.isfinite(y).all() and torch.isfinite(h).all()
    cut = {k: v[1:, :5] if v.dim() > 2 else v for k, v in p.items()}
    _, before = fw.selective_scan(*cut.values(), **dict(o, h0=o["h0"][1:], gate=o["gate"][1:, :5]))
    assert torch.equal(h[1:], before)
    p["dt"] = p["dt"].clamp(min=-100.0)  # for the oracle: a step of exp(-100) is as good as none
    want = _oracle(p, o).forward()
    _close(y, want["y"], "y")
    _close(h, want["h"], "h")
    out = fw.selective_scan_step(*(v[:, 20] if v.dim() > 2 else v for v in {**p, "dt": torch.full_like(p["dt"], float("-inf"))}.values()),
                                 h.clone(), dt_bias=o["dt_bias"])
    assert torch.isfinite(out).all()


def test_gates_far_from_zero():
    """silu and its slope at the ends: 0 and z, without NaN."""
    p, o, n = _make(1, 40, 1, 8, 4, F32, seed=23)
    o["gate"][0, :20] = -200.0
    o["gate"][0, 20:] = 200.0
    _both(p, o, n)
    y, _ = fw.selective_scan(*p.values(), **o)
    assert not y[0, :20].any()
