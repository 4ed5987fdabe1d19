"""Digits that the selective state space block keeps: decays that forget, rates without end, slopes far from zero, long sums and
rows behind a length.  Every tolerance counts half steps, U = 2^-24 of a value, and is stated beside its test."""
import numpy as np
import pytest
import torch

import newton_solve_nonlinear_b200 as fw
from oracle import bounds
from tests.test_gpu_selective_scan import BF16, F32

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _relative(got, want, steps, what):
    """got is within `steps` half steps of want, element by element, and its rounding to bf16."""
    tol = steps * U + (2.0 ** -8 if got.dtype == BF16 else 0.0)
    worst = float(((got.double() - want).abs() / want.abs()).max())
    assert worst <= tol, f"{what}: {worst:.3g} of the value, {tol:.3g} allowed"


def _forgetting(B, T, G, per, N, dtype, seed):
    """A step of 1 and rates of 8 to 30: each token replaces the state.  All is positive, so that no sum cancels; inputs lie
    between 1e-5 and 1e4, so that a small one often follows a large one."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = lambda lo, hi, *s: lo + (hi - lo) * torch.rand(*s, device="cuda", generator=g)
    D = G * per
    p = dict(x=10 ** u(-5, 4, B, T, D), dt=torch.ones(B, T, D, device="cuda"), a=-u(8, 30, D, N), b=u(0.5, 1.5, B, T, G, N),
             c=u(0.5, 1.5, B, T, G, N))
    p = {k: v if k == "a" else v.to(dtype) for k, v in p.items()}
    return p, u(1, 100, B, D, N), u(0.5, 1.5, B, T, D).to(dtype), u(0.5, 1.5, B, D, N)


def _forgetting64(p, h0, dy, dh):
    """The formulas in 64 bits: the states, y and every gradient."""
    x, a, dy, h, P = p["x"].double(), p["a"].double(), dy.double(), h0.double(), dh.double()
    B, T, D = x.shape
    G, N = p["b"].shape[2:]
    b, c = (p[k].double().repeat_interleave(D // G, dim=2) for k in "bc")
    w, hs = torch.exp(a), [h]
    for t in range(T):
        hs.append(w * hs[-1] + x[:, t, :, None] * b[:, t])
    y = torch.stack([(c[:, t] * hs[t + 1]).sum(-1) for t in range(T)], 1)
    da, out = torch.zeros_like(a), dict(dx=[], ddt=[], db=[], dc=[])
    shared = lambda v: v.reshape(B, G, D // G, N).sum(2)
    for t in reversed(range(T)):
        g = P + dy[:, t, :, None] * c[:, t]
        gb = (g * b[:, t]).sum(-1)
        out["dc"].insert(0, shared(dy[:, t, :, None] * hs[t + 1]))
        out["db"].insert(0, shared(g * x[:, t, :, None]))
        out["dx"].insert(0, gb)
        P = w * g
        da += (P * hs[t]).sum(0)
        out["ddt"].insert(0, (a * P * hs[t]).sum(-1) + x[:, t] * gb)
    return y, hs[-1], dict({k: torch.stack(v, 1) for k, v in out.items()}, da=da, dh0=P)


# one token and a few; segments of time; each width of a full card: 104 groups give 104 CTAs, which take four states a thread
FORGETTING = [(2, 1, 1, 6, 16), (1, 5, 1, 3, 2), (2, 300, 2, 20, 16), (1, 200, 1, 9, 64), (1, 9, 104, 1, 3), (1, 20, 104, 1, 7),
              (1, 20, 104, 2, 16), (2, 17, 52, 66, 16), (1, 20, 104, 1, 30), (1, 20, 104, 2, 64)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", FORGETTING)
def test_a_decay_that_forgets_keeps_its_own_digits(size, dtype):
    """exp(z) is off by U for each of z's two roundings and the constant's, times |z| <= 30, and by ex2's four U: 94 U; the
    product and the sum round twice more.  What a token inherits is at most e^-8 of errors like these once more, so 100 U
    hold for a state and for P, 200 U for their product, and every sum of n positive terms adds n U."""
    B, T, G, per, N = size
    p, h0, dy, dh = _forgetting(*size, dtype, seed=N)
    y, h, kept = fw.selective_scan(*p.values(), softplus=False, h0=h0, keep=True)
    wy, wh, want = _forgetting64(p, h0, dy, dh)
    _relative(h, wh, 110, "h")
    _relative(y, wy, 110 + N, "y")
    for given in (kept, None):
        g = fw.selective_scan_backward(*p.values(), dy, softplus=False, h0=h0, dh=dh, kept=given)
        for k, steps in dict(dh0=110, da=220 + T + B, dx=110 + N, db=110 + per, dc=110 + per).items():
            _relative(g[k], want[k], steps, k)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [(2, 1, 1, 6, 16), (1, 2, 1, 5, 64), (1, 2, 104, 2, 16)])
def test_a_step_s_gradient_through_decays_that_forget(size, dtype):
    """Without inputs ddt is the sum of a P h alone, of one sign: 200 U for P h, one for the rate and N for the sum."""
    p, h0, dy, dh = _forgetting(*size, dtype, seed=3)
    p["x"].zero_()
    g = fw.selective_scan_backward(*p.values(), dy, softplus=False, h0=h0, dh=dh)
    _relative(g["ddt"], _forgetting64(p, h0, dy, dh)[2]["ddt"], 230 + size[-1], "ddt")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,G,per,N", [(1, 1, 5, 1), (3, 2, 21, 5), (2, 1, 300, 16), (5, 1, 40, 64)])
def test_a_step_that_forgets(B, G, per, N, dtype):
    """As above, for one token of each sequence."""
    p, h0, dy, dh = _forgetting(B, 1, G, per, N, dtype, seed=4)
    q = {k: v if k == "a" else v[:, 0] for k, v in p.items()}
    state = h0.clone()
    y = fw.selective_scan_step(*q.values(), state, softplus=False)
    wy, wh, _ = _forgetting64(p, h0, dy, dh)
    _relative(state, wh, 110, "state")
    _relative(y[:, None], wy, 110 + N, "y")


@pytest.mark.parametrize("rate", [float("-inf"), -3e38])
@pytest.mark.parametrize("size", [(3, 13, 1, 6, 16), (3, 300, 1, 5, 9), (3, 13, 35, 2, 16)])
def test_rates_without_end(size, rate):
    """A rate of -inf forgets at every token, and only there: the places behind a length, the empty segments and tokens of
    step zero (softplus of -inf) decay nothing.  -1e30 takes the same steps with finite products, to the same bits."""
    B, T, G, per, N = size
    D = G * per
    g = torch.Generator(device="cuda").manual_seed(9)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)
    p = dict(x=n(B, T, D), dt=n(B, T, D), a=-torch.exp(n(D, N)), b=n(B, T, G, N), c=n(B, T, G, N))
    p["a"][:, ::2] = -1e30
    o = dict(h0=n(B, D, N), lengths=torch.tensor([T, 0, min(T - 2, 70)], dtype=torch.int32, device="cuda"))
    dy, dh = n(B, T, D), n(B, D, N)

    def run(a):
        q = dict(p, a=a)
        y, h, kept = fw.selective_scan(*q.values(), keep=True, **o)
        back = fw.selective_scan_backward(*q.values(), dy, dh=dh, **o)
        q["dt"] = p["dt"].clone()
        q["dt"][:, 5:8] = float("-inf")
        z, k = fw.selective_scan(*q.values(), **o)
        pool = o["h0"].clone()
        one = {k: v if k == "a" else v[:, 5] for k, v in q.items()}
        out = fw.selective_scan_step(*one.values(), pool)
        return dict(back, y=y, h=h, z=z, k=k, step=out, pool=pool)

    want, got = run(p["a"]), run(torch.where(p["a"] == -1e30, rate, p["a"]))
    for k, v in want.items():
        if v is not None:
            assert torch.isfinite(v).all() and torch.equal(got[k], v), k
    assert torch.equal(got["pool"], o["h0"]) and torch.equal(got["h"][1], o["h0"][1])
    assert torch.equal(got["dh0"][1], dh[1])


def test_growth_past_fp32_of_a_state_that_is_zero():
    """Rates above zero over segments of time whose growth, exp(a times the segment's steps), passes fp32: a state that is
    zero stays zero, as it does token by token."""
    T, D, N = 6000, 3, 4
    x, a = torch.zeros(1, T, D, device="cuda"), torch.full((D, N), 3.0, device="cuda")
    dt, b = torch.ones_like(x), torch.ones(1, T, 1, N, device="cuda")
    x[:, -1] = 2.0
    y, h = fw.selective_scan(x, dt, a, b, b, softplus=False)
    assert not y[:, :-1].any() and (y[:, -1] == 2.0 * N).all() and (h == 2.0).all()
    dy = torch.zeros_like(x)
    dy[:, 0] = 3.0
    x.zero_()
    g = fw.selective_scan_backward(x, dt, a, b, b, dy, softplus=False, h0=torch.zeros(1, D, N, device="cuda"))
    assert (g["dx"][:, 0] == 3.0 * N).all() and not g["dx"][:, 1:].any() and not g["da"].any()
    torch.testing.assert_close(g["dh0"], torch.full_like(g["dh0"], 3.0 * float(np.exp(3.0))), rtol=20 * U, atol=0)


def test_steps_far_from_zero():
    """One token of one state from zero leaves h = softplus(dt): off by 16 U of it at most, at exp(-85) as near zero."""
    dt = torch.cat([torch.arange(-85, 20, 0.37), torch.arange(-1, 1, 0.01)]).cuda()
    D = dt.numel()
    one = torch.ones(1, 1, D, device="cuda")
    b = torch.ones(1, 1, 1, 1, device="cuda")
    _, h = fw.selective_scan(one, dt.reshape(1, 1, D), torch.full((D, 1), -1e4, device="cuda"), b, b)
    z = dt.double()
    want = z.clamp(min=0) + torch.log1p(torch.exp(-z.abs()))
    assert float(((h.flatten().double() - want).abs() / want).max()) <= 16 * U


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_slopes_far_from_zero(dtype):
    """dweight and dbias are fp32 whatever the inputs' type.  One token, one tap and dy = 1: the bias' gradient is silu's slope
    at x, which bf16 holds exactly, and the tap's is that times x.  bounds.silu_slope_bound counts what fp32 makes of it."""
    x = torch.cat([-torch.arange(1, 85, 0.5), torch.arange(0, 20, 0.5)]).to(dtype).cuda()
    D = x.numel()
    w = torch.zeros(D, 4, device="cuda")
    w[:, 3] = 1.0
    g = fw.causal_conv_backward(x.reshape(1, 1, D), w, torch.ones(1, 1, D, device="cuda", dtype=dtype), torch.zeros(D, device="cuda"))
    z = x.double().cpu().numpy()
    want, tol = bounds.silu_slope(z), bounds.silu_slope_bound(z).e
    off = np.abs(g["dbias"].double().cpu().numpy() - want)
    assert (off <= tol + 1e-37).all(), float((off / (tol + 1e-37)).max())
    off = np.abs(g["dweight"][:, 3].double().cpu().numpy() - want * z)
    assert (off <= (tol + U * np.abs(want)) * np.abs(z) + 1e-35).all()
    assert not g["dweight"][:, :3].any()


def _sum_is_exact_to(got, want, steps, what):
    off = float((got.double() - want).abs().max() / abs(want))
    assert off <= steps * U, f"{what}: {off / U:.0f} half steps, {steps:.0f} allowed"


def test_long_sums_of_the_scan_s_parameters():
    """dskip, ddt_bias and da over 65536 tokens that are all alike: an fp32 chain loses the same part of each term, again and
    again: n of them by up to n / 2 half steps of the sum.  Pieces of at most 64 tokens lose 32 U, the eight chains of T / 512
    of them T / 1024 U, the sums over chains and rows 40 U; a term is a product of up to four factors, 8 U.  (100 groups: a card full of CTAs, so time is not split.)"""
    T, D = 65536, 100
    x, v = 0.63, 0.77
    full = lambda *s, value: torch.full(s, value, device="cuda")
    a = full(D, 1, value=-1e4)  # a token replaces the state
    one = full(1, T, D, 1, value=1.0)
    g = fw.selective_scan_backward(full(1, T, D, value=x), full(1, T, D, value=1.0), a, one, one, full(1, T, D, value=v),
                                   skip=full(D, value=0.0), dt_bias=full(D, value=0.0), softplus=False)
    term = float(np.float32(x)) * float(np.float32(v))
    steps = 32 + T / 1024 + 40 + 8
    _sum_is_exact_to(g["dskip"], T * term, steps, "dskip")
    _sum_is_exact_to(g["ddt_bias"], T * term, steps, "ddt_bias")


def test_long_sums_over_sequences():
    """The same over 2^21 sequences of one token: 32 warps take the rows of partial sums, pieces of 64 in chains of 16, 8 U and two
    more, and a chain of pieces, B / 4096 U; 8 U for the warps' sum, 8 U for a term."""
    B = 1 << 21
    full = lambda *s, value: torch.full(s, value, device="cuda")
    one, p = full(B, 1, 1, 1, value=1.0), full(1, value=0.0)
    g = fw.selective_scan_backward(full(B, 1, 1, value=0.63), full(B, 1, 1, value=1.0), full(1, 1, value=-1e4), one, one,
                                   full(B, 1, 1, value=0.77), skip=p, dt_bias=p, softplus=False)
    term = float(np.float32(0.63)) * float(np.float32(0.77))
    steps = 10 + B / 4096 + 8 + 8
    _sum_is_exact_to(g["dskip"], B * term, steps, "dskip")
    _sum_is_exact_to(g["ddt_bias"], B * term, steps, "ddt_bias")


@pytest.mark.parametrize("B,T,D", [(1, 16384, 32768), (16, 4096, 32768), (3, 16384, 32767)])
def test_long_sums_of_the_convolution_s_parameters(B, T, D):
    """As above for taps and bias: a thread has whole sequences, or 2048 tokens and more of one.  Pieces of at most 64 tokens
    lose 32 U and a chain of them, B T / 8 tokens to a thread at most, B T / 1024 U; 40 U for the sums over a CTA's threads and
    over the CTAs, and for the product.  (x and dy are one value, expanded.)"""
    x = torch.full((1, 1, 1), 0.63, device="cuda").expand(1, 1, D).contiguous().expand(B, T, D)
    dy = torch.full((D,), 0.77, device="cuda").expand(B, T, D)
    g = fw.causal_conv_backward(x, torch.zeros(D, 4, device="cuda"), dy, torch.zeros(D, device="cuda"), act="none")
    assert not g["dx"].any()
    x, v = float(np.float32(0.63)), float(np.float32(0.77))
    steps = 32 + B * T / 1024 + 40
    _sum_is_exact_to(g["dbias"], B * T * v, steps, "dbias")
    for j in range(4):
        _sum_is_exact_to(g["dweight"][:, j], B * (T - 3 + j) * x * v, steps, f"tap {j}")


@pytest.mark.parametrize("rows,C,teams", [(1 << 22, 8, 8), (1 << 20, 1024, 1), (1 << 18, 4096, 1), (1 << 18, 8192, 1), (1 << 17, 9216, 1),
                                          (1 << 16, 32769, 8)])
def test_long_sums_of_the_norm_s_parameters(rows, C, teams):
    """As above for weight and bias: at least 148 CTAs of `teams` each take a row at a time, add up pieces of at most 64 rows, 32 U,
    and a chain of the pieces; 40 U for the sums over the teams."""
    r, dy = (torch.full((rows, C), value, device="cuda") for value in (0.63, 0.1))
    stats = torch.tensor([0.0, 1.0], device="cuda").repeat(rows, 1)
    g = fw.layer_norm_backward(r, stats, dy, torch.ones(C, device="cuda"), torch.zeros(C, device="cuda"), rms=True)
    steps = 32 + rows / 148 / teams / 128 + 40 + 1
    want = float(np.float32(0.1))
    _sum_is_exact_to(g["dbias"], rows * want, steps, "dbias")
    _sum_is_exact_to(g["dweight"], rows * want * float(np.float32(0.63)), steps, "dweight")


@pytest.mark.parametrize("C", [24, 33, 500, 1100, 9000, 33000])
@pytest.mark.parametrize("rms", [False, True])
def test_rows_behind_a_length_are_zero_whatever_the_weight(C, rms):
    """A weight or bias that is not finite reaches the rows that count, and no others."""
    g = torch.Generator(device="cuda").manual_seed(C)
    x, res = (torch.randn(2, 3, C, device="cuda", generator=g) for _ in range(2))
    w, b = torch.ones(C, device="cuda"), torch.zeros(C, device="cuda")
    w[1], w[C - 1], b[2] = float("inf"), float("nan"), float("nan")
    y, r, stats = fw.layer_norm(x, w, b, residual=res, rms=rms, lengths=torch.tensor([1, 0], dtype=torch.int32, device="cuda"))
    assert not y[0, 1:].any() and not y[1].any() and not r[0, 1:].any() and not r[1].any()
    assert torch.isinf(y[0, 0, 1]) and torch.isnan(y[0, 0, C - 1]) and torch.isnan(y[0, 0, 2])
