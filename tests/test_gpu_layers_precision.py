"""How exact linear attention's state and group norm's activations are, by inputs that leave nothing else to round."""
import math

import numpy as np
import pytest
import torch

import newton_solve_nonlinear_b200 as fw
from oracle import group_norm as gn

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS24, EPS23 = 2.0 ** -24, 2.0 ** -23


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T,t,tol", [(6, 0, 2.0 ** -20), (128, 100, 2.0 ** -20), (1024, 890, 2.0 ** -19)])
def test_state_products_are_exact_to_fp32(T, t, tol, dk, dv):
    """bf16 operands, all tokens zero but one: the state is w k v^T with one weight w.

    w is within 2 ulp, 2^-22; y = w v is rounded once, 2^-24, and its three bf16 terms are exact (24 bits); their products
    with k are exact in fp32 and added in two steps, each within an ulp, 2^-23: 2.25 2^-22 < 2^-20 in all.  With 1024
    tokens of one head time is split into segments of 128: the state of the second but last one is multiplied by one
    more weight, 1.25 2^-22 more.  Two terms would leave up to 2^-16 of y."""
    g = torch.Generator("cuda").manual_seed(dk + dv + T)
    q, k, v = (torch.zeros(1, T, 1, d, dtype=BF16, device="cuda") for d in (dk, dk, dv))
    k[0, t, 0].normal_(generator=g)
    v[0, t, 0].normal_(generator=g)
    ld = torch.tensor([-0.017], device="cuda")
    _, s = fw.linear_attention(q, k, v, ld)
    w = torch.exp(ld.double() * (T - 1 - t))
    want = k[0, t, 0].double()[:, None] * (w * v[0, t, 0].double())[None]
    assert bool(((s[0, 0].double() - want).abs() <= tol * want.abs()).all())
    # what these inputs would show of a kernel with two terms
    y = (w.float() * v[0, t, 0].float())
    u0 = y.to(BF16).float()
    two = u0 + (y - u0).to(BF16).float()
    assert float(((y - two).abs() / y.abs()).max()) > 2.0 ** -18 > tol


def _points(low, high):
    z = np.concatenate([np.linspace(low, high, 1500), np.linspace(-3.0, 3.0, 547), [0.0]]).astype(np.float32)
    return torch.from_numpy(z[: 2048]).cuda()


def _act_error(z, act):
    """(value, its error, slope, its error) of the activation in fp32.

    __expf(x) is within 2 + floor(|1.173 x|) ulp, the approximate reciprocal within one, each of 2^-23; normcdff within 5.
    The sigmoid s = 1 / (1 + E) takes E's error by 1 - s, and the value and the slope, s + z s (1 - s), where 1 - s is
    within the absolute error of s, a rounding for each operation."""
    if act == "silu":
        s = 1 / (1 + np.exp(-z))
        es = s * ((1 - s) * (2 + 1.173 * np.abs(z)) + 1 + 0.5) * EPS23
        a = z * s
        ea = np.abs(z) * es + EPS24 * np.abs(a)
        slope = s + a * (1 - s)
        return a, ea, slope, es + ea * (1 - s) + np.abs(a) * (es + EPS24 * (1 - s)) + EPS24 * (np.abs(slope) + np.abs(a * (1 - s)))
    p = gn._phi(z)
    h = z * z / 2
    d = np.abs(z) * np.exp(-h) / math.sqrt(2 * math.pi)
    slope = gn.slope(z, "gelu")
    # the exponent is rounded twice, z times the constant twice (the constant itself once)
    return z * p, 5.5 * EPS23 * np.abs(z * p), slope, d * ((2 + 1.173 * h) * EPS23 + 2 * h * EPS24 + 2 * EPS24) + 5 * EPS23 * p + EPS24 * np.abs(slope)


@pytest.mark.parametrize("act,low,high", [("silu", -80.0, 80.0), ("gelu", -12.0, 12.0)])
@pytest.mark.parametrize("shape", [(1, 1, 2048), (1, 3, 2048)])
def test_activations_far_from_zero(shape, act, low, high):
    """With a weight of zero z is the bias itself, and y, dgate and dbias are the activation and its slope."""
    N, S, C = shape
    z = _points(low, high)
    zero, one = torch.zeros(C, device="cuda"), torch.ones(C, device="cuda")
    x = torch.randn(N, S, C, device="cuda")
    zn = z.double().cpu().numpy()
    a, ea, s, es = _act_error(zn, act)
    floor = 1e-37  # results below are subnormal
    near = lambda got, want, tol: np.all(np.abs(got.double().cpu().numpy() - want) <= tol + floor)
    y, stats = fw.group_norm(x, 4, zero, z, act=act)
    assert all(near(y[0, i], a, ea) for i in range(S))
    dy = torch.zeros_like(x)
    dy[0, 0] = 1
    assert near(fw.group_norm_backward(x, stats, dy, 4, zero, z, act=act)["dbias"], s, es)
    gate = z.expand(N, S, C).contiguous()
    y, stats = fw.group_norm(x, 4, zero, one, act=act, gate=gate)
    assert all(near(y[0, i], a, ea) for i in range(S))
    dgate = fw.group_norm_backward(x, stats, torch.ones_like(x), 4, zero, one, act=act, gate=gate)["dgate"]
    assert all(near(dgate[0, i], s, es) for i in range(S))


def _state_and_last_output(q, k, v, ld, s0):
    """In fp64: the state after all tokens and the last token's output, [B, H, dk, dv] and [B, H, dv]."""
    B, T, H, dk = q.shape
    s = torch.empty(B, H, dk, v.shape[3], dtype=torch.float64, device="cuda")
    age = torch.arange(T - 1, -1, -1, dtype=torch.float64, device="cuda")
    for h in range(H):
        w = torch.exp(age * ld[h].double())[None, :, None]
        s[:, h] = (k[:, :, h].double() * w).transpose(1, 2) @ v[:, :, h].double()
        s[:, h] += torch.exp(T * ld[h].double()) * s0[:, h].double()
    return s, dk ** -0.5 * torch.einsum("bhk,bhkv->bhv", q[:, -1].double(), s)


@pytest.mark.parametrize("decay", [-2.4e-4, -1e-5, -1e-6])
@pytest.mark.parametrize("B,T,H,d", [(2, 8192, 80, 32), (1, 8192, 1, 64), (2, 16384, 37, 64)])
def test_slow_decays_keep_fp32(B, T, H, d, decay):
    """fp32, memories of thousands of tokens, one sweep or segments of time.

    What is carried from chunk to chunk or segment to segment, K of them, is rounded once each time: half an ulp at most,
    2^-23 / sqrt(12) in the root mean square, independent of one another, so sqrt(K) of that for the whole, less as the
    state grows.  K is 512 at most here, 7.8e-7.  A weight that is rounded before it is carried along would be off by K
    times the same rounding, and sums of all products one by one by sqrt(T) of it.  o adds d roundings of its own products
    and those of its chunk.  2^-20 is 9.5e-7."""
    g = torch.Generator("cuda").manual_seed(T + H)
    q, k, v = (torch.randn(B, T, H, d, device="cuda", generator=g) for _ in range(3))
    s0 = torch.randn(B, H, d, d, device="cuda", generator=g)
    ld = decay * torch.linspace(0.7, 1.3, H, device="cuda")
    o, s = fw.linear_attention(q, k, v, ld, s0=s0)
    ws, wo = _state_and_last_output(q, k, v, ld, s0)
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())
    assert rel(s, ws) <= 2.0 ** -20
    assert rel(o[:, -1], wo) <= 2.0 ** -20


@pytest.mark.parametrize("decay", [-2.4e-4, -1e-5, -1e-6])
@pytest.mark.parametrize("B,T,H,dk,dv", [(2, 8192, 80, 32, 64), (2, 16384, 80, 64, 64), (2, 16384, 74, 128, 100),
                                         (1, 16384, 1, 64, 128), (1, 65536, 8, 64, 64)])
def test_slow_decays_keep_the_state_of_bf16_operands(B, T, H, dk, dv, decay):
    """As above for the state, whose products are exact and whose chunks have 128 tokens: K is 128 at most in one sweep."""
    g = torch.Generator("cuda").manual_seed(T + H)
    q, k, v = (torch.randn(B, T, H, d, device="cuda", generator=g).to(BF16) for d in (dk, dk, dv))
    s0 = torch.randn(B, H, dk, dv, device="cuda", generator=g)
    ld = decay * torch.linspace(0.7, 1.3, H, device="cuda")
    _, s = fw.linear_attention(q, k, v, ld, s0=s0)
    ws, _ = _state_and_last_output(q, k, v, ld, s0)
    assert float((s.double() - ws).norm() / ws.norm()) <= 2.0 ** -20
    # backward: the same of the state carried in reversed time, dL/ds0
    do = torch.randn(B, T, H, dv, device="cuda", generator=g).to(BF16)
    got = fw.linear_attention_backward(q, k, v, ld, do, s0=s0, ds=s0)["ds0"]
    age = torch.arange(1, T + 1, dtype=torch.float64, device="cuda")
    want = torch.empty_like(ws)
    for h in range(H):
        w = torch.exp(age * ld[h].double())[None, :, None]
        want[:, h] = dk ** -0.5 * ((q[:, :, h].double() * w).transpose(1, 2) @ do[:, :, h].double())
        want[:, h] += torch.exp(T * ld[h].double()) * s0[:, h].double()
    assert float((got.double() - want).norm() / want.norm()) <= 2.0 ** -20


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("decay", [-0.05, -0.3, -0.6, -5.0, -50.0])
@pytest.mark.parametrize("T", [333, 700, 1100])
def test_a_state_that_decays_to_nothing(T, decay, dtype):
    """No inputs but a start state (forward) or a last gradient (backward), which is carried alone: g^T of it, by factors
    that are each within 2 ulp of g^n and one rounding for each of up to 36 chunks: 36 * 2.5 * 2^-23 < 2^-16, relative
    however small it gets."""
    B, H, d = 2, 4, 64
    q, k, v, do = (torch.zeros(B, T, H, d, dtype=dtype, device="cuda") for _ in range(4))
    s0 = torch.randn(B, H, d, d, device="cuda", generator=torch.Generator("cuda").manual_seed(T))
    ld = torch.full((H,), decay, device="cuda")
    lengths = torch.tensor([T, T - 130], dtype=torch.int32, device="cuda")
    _, s = fw.linear_attention(q, k, v, ld, s0=s0, lengths=lengths)
    ds0 = fw.linear_attention_backward(q, k, v, ld, do, s0=s0, ds=s0, lengths=lengths)["ds0"]
    want = torch.exp(lengths.double() * ld[0].double())[:, None, None, None] * s0.double()
    for got in (s, ds0):
        assert bool(((got.double() - want).abs() <= 2.0 ** -16 * want.abs() + 2.0 ** -126).all())


@pytest.mark.parametrize("decay,tol", [(-1e-6, 2.0 ** -12), (-3.3e-5, 2.0 ** -18), (-1e-3, 2.0 ** -18)])
def test_slow_decays_token_by_token(decay, tol):
    """4096 single-token steps without inputs: the state is g^4096 of what it was.  A step rounds it once, 2^-23 / sqrt(12)
    in the root mean square at most: sqrt(4096) of that is 2.2e-6 < 2^-18.  A weight of one fp32 would be off by up to 2^-25
    each time, all in one direction: 1.2e-4.

    That takes roundings that differ from step to step.  A step takes |decay| 2^23 to |decay| 2^24 ulp off the state, which
    changes by |decay| of itself: at -1e-3 by 8 ulp and more, at -3.3e-5 by 0.009 ulp, so 37 ulp over the steps.  At -1e-6 8
    to 17 ulp change by less than 0.07 ulp in all 4096 steps: they are rounded alike, by up to half an ulp, 4096 2^-24."""
    B, H, d, n = 2, 3, 32, 4096
    state = torch.randn(B, H, d, d, device="cuda", generator=torch.Generator("cuda").manual_seed(11))
    start, zero = state.double(), torch.zeros(B, H, d, device="cuda")
    ld = decay * torch.tensor([0.77, 1.0, 1.23], device="cuda")
    for _ in range(n):
        fw.linear_attention_step(zero, zero, zero, ld, state)
    want = torch.exp(n * ld.double())[None, :, None, None] * start
    off = (state.double() - want).flatten(2).norm(dim=2) / want.flatten(2).norm(dim=2)
    assert float(off.max()) <= tol


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("decay,tol", [(-1e-6, 2.0 ** -16), (-3.3e-5, 2.0 ** -18), (-1e-3, 2.0 ** -18)])
def test_slow_decays_token_by_token_with_inputs(decay, tol, dtype):
    """As above with tokens that differ, so that the roundings do: two a step (the product's and the state's, the first one
    smaller), sqrt(4096) of them, and less while the state grows: 2^-18.

    Products of bf16 values have 16 bits, multiples of a state's ulp once it is some 2^6 large, so that only what a step
    takes off is rounded.  It changes with the state by |decay| |k v|, at -1e-6 by some 0.1 ulp (2^-17) a step, and wanders
    over half an ulp in (0.5 / 0.1)^2 = 25 steps, which are rounded alike: sqrt(25) 2.2e-6 < 2^-16 there."""
    B, H, d, n = 2, 3, 32, 4096
    g = torch.Generator("cuda").manual_seed(12)
    q, k, v = (torch.randn(B, n, H, d, device="cuda", generator=g).to(dtype) for _ in range(3))
    state = torch.randn(B, H, d, d, device="cuda", generator=g)
    ld = decay * torch.tensor([0.77, 1.0, 1.23], device="cuda")
    want, _ = _state_and_last_output(q, k, v, ld, state)
    for t in range(n):
        fw.linear_attention_step(q[:, t], k[:, t], v[:, t], ld, state)
    off = (state.double() - want).flatten(2).norm(dim=2) / want.flatten(2).norm(dim=2)
    assert float(off.max()) <= tol
