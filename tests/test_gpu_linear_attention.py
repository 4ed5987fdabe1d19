"""Linear attention with a decay for each head on the GPU against the fp64 recurrence (oracle/linear_attention.py).

Tolerances are elementwise, against the same sums taken over absolute values (``mag``), which bounds every
rounding: a path from an input to an output holds at most n = dk + dv + T + 64 fp32 roundings (dot products, the
weights, the chunk sums, the carried state), so fp32 results are within n 2^-24 mag.  With bf16 operands each
product for o (dq, dk, dv) has one factor, the weighted score or the state's copy, rounded to bf16: 2^-8 mag more,
and the result itself is rounded: 2^-8 |result|.  States stay fp32.
"""
import numpy as np
import pytest
import torch

import newton_solve_nonlinear_b200 as fw
from newton_solve_nonlinear_b200 import binding
from oracle import linear_attention as oracle

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _make(B, T, H, Hkv, dk, dv, dtype, seed=0, start=True, decay=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, dt=dtype: torch.randn(*s, device="cuda", generator=g).to(dt)
    ld = torch.linspace(-0.01, -1.0, H, device="cuda") if decay is None else torch.tensor(decay, device="cuda")
    return dict(q=n(B, T, H, dk), k=n(B, T, Hkv, dk), v=n(B, T, Hkv, dv), log_decay=ld,
                s0=n(B, H, dk, dv, dt=F32) if start else None), n


def _close(got, want, mag, n, dtype, what):
    got = _np(got)
    assert np.all(np.isfinite(got)), what
    tol = n * 2.0 ** -24 * mag + 1e-30
    if dtype == BF16:
        tol = tol + 2.0 ** -8 * (mag + np.abs(want))
    worst = float(np.max(np.abs(got - want) / tol)) if got.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times the tolerance"


def _check_forward(a, lengths=None, scale=None, **kw):
    q, k, v, ld, s0 = (a[n] for n in ("q", "k", "v", "log_decay", "s0"))
    B, T, H, dk = q.shape
    dv, sc = v.shape[3], dk ** -0.5 if scale is None else scale
    o, s = fw.linear_attention(q, k, v, ld, s0=s0, lengths=lengths, scale=scale, **kw)
    ln = None if lengths is None else lengths.tolist()
    q, k, v, s0 = _np(q), _np(k), _np(v), _np(s0)
    if ln is not None:  # what stands behind the lengths is not read
        for b, L in enumerate(ln):
            q[b, max(L, 0):], k[b, max(L, 0):], v[b, max(L, 0):] = 0, 0, 0
    ld = _np(ld)
    wo, ws = oracle.forward(q, k, v, ld, s0, ln, sc)
    mo, ms = oracle.forward(abs(q), abs(k), abs(v), ld, None if s0 is None else abs(s0), ln, abs(sc))
    n = dk + dv + T + 64
    _close(o, wo, mo, n, a["q"].dtype, "o")
    _close(s, ws, ms, n, F32, "state")
    return o, s


SIZES = [
    # B, T, H, Hkv, dk, dv
    (1, 1, 1, 1, 1, 1), (2, 1, 4, 2, 64, 64), (1, 2, 3, 3, 5, 7), (3, 31, 2, 1, 16, 16), (2, 32, 2, 2, 64, 128),
    (2, 33, 4, 4, 128, 128), (1, 127, 6, 2, 80, 96), (2, 128, 2, 2, 128, 64), (1, 129, 3, 1, 33, 65),
    (2, 300, 2, 1, 64, 64), (1, 1025, 2, 2, 96, 128), (5, 257, 4, 1, 127, 1), (1, 640, 8, 8, 1, 127),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", SIZES)
def test_forward(size, dtype):
    a, _ = _make(*size, dtype)
    _check_forward(a)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [(2, 150, 4, 2, 64, 64), (1, 600, 2, 2, 128, 48)])
def test_forward_without_start_state_and_with_other_scale(size, dtype):
    a, _ = _make(*size, dtype, start=False)
    _check_forward(a, scale=1.0)
    _check_forward(a, scale=-0.3)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward_decays_from_none_to_all(dtype):
    a, _ = _make(2, 400, 6, 6, 32, 64, dtype, decay=[0.0, -1e-4, -0.5, -8.0, -200.0, float("-inf")])
    _check_forward(a)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,lengths", [(200, [200, 0, 1, 129, 128]), (1500, [0, 1499, 600, 1025, 7]),
                                       (70, [-3, 71, 69, 1 << 30, 33])])
def test_forward_padded_batch(T, lengths, dtype):
    a, n = _make(5, T, 4, 2, 64, 48, dtype)
    for b, L in enumerate(lengths):
        L = min(max(L, 0), T)
        for x in ("q", "k", "v"):
            a[x][b, L:] = float("nan") if b % 2 else float("inf")
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o, s = fw.linear_attention(a["q"], a["k"], a["v"], a["log_decay"], s0=a["s0"], lengths=ln)
    o2, s2 = _check_forward(a, lengths=ln.clamp(0, T))
    assert torch.equal(o, o2) and torch.equal(s, s2)
    for b, L in enumerate(lengths):
        L = min(max(L, 0), T)
        assert not o[b, L:].any()
        if L == 0:
            assert torch.equal(s[b], a["s0"][b])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward_strided_views(dtype):
    """q, k, v as views of one projected tensor, heads before time, and shared by stride 0."""
    g = torch.Generator(device="cuda").manual_seed(3)
    B, T, H, Hkv, dk, dv = 2, 140, 4, 2, 64, 64
    x = torch.randn(B, T, (H + 2 * Hkv) * 64 + 3, device="cuda", generator=g).to(dtype)
    q, k, v = x[..., :256].unflatten(-1, (H, 64)), x[..., 256:384].unflatten(-1, (2, 64)), x[..., 384:512].unflatten(-1, (2, 64))
    ld = torch.full((H,), -0.05, device="cuda")
    _check_forward(dict(q=q, k=k, v=v, log_decay=ld, s0=None))
    _check_forward(dict(q=x[..., 1:257].unflatten(-1, (H, 64)), k=k, v=v, log_decay=ld, s0=None))
    t = lambda y: y.transpose(1, 2).contiguous().transpose(1, 2)
    _check_forward(dict(q=t(q), k=t(k), v=t(v), log_decay=ld, s0=None))
    one = k[:, :, :1].contiguous().expand(B, T, H, 64)
    _check_forward(dict(q=q, k=one, v=v[:, :, :1].contiguous().expand(B, T, H, 64), log_decay=ld, s0=None))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward_long_sequence_in_parts_equals_whole(dtype):
    """A long prompt in one call and in two calls that hand the state on; sampled against the fp64 sum."""
    a, _ = _make(1, 20011, 2, 1, 64, 64, dtype, decay=[-1e-3, -0.02])
    q, k, v, ld, s0 = (a[n] for n in ("q", "k", "v", "log_decay", "s0"))
    o, s = fw.linear_attention(q, k, v, ld, s0=s0)
    cut = 7003
    o1, s1 = fw.linear_attention(q[:, :cut], k[:, :cut], v[:, :cut], ld, s0=s0)
    o2, s2 = fw.linear_attention(q[:, cut:], k[:, cut:], v[:, cut:], ld, s0=s1, out=(torch.empty_like(o[:, cut:]), s1))
    assert s2 is s1  # the state replaced in place
    T, dk = q.shape[1], 64
    K, V = k.double()[0, :, 0], v.double()[0, :, 0]
    for h in range(2):
        for t in (0, cut - 1, cut, 12345, T - 1):
            w = torch.exp((t - torch.arange(t + 1, device="cuda", dtype=torch.float64)) * ld[h].double())
            p = w * (K[:t + 1] @ q[0, t, h].double())
            want = dk ** -0.5 * (p @ V[:t + 1] + torch.exp((t + 1) * ld[h].double()) * q[0, t, h].double() @ s0[0, h].double())
            mag = dk ** -0.5 * (p.abs() @ V[:t + 1].abs() + torch.exp((t + 1) * ld[h].double())
                                * q[0, t, h].double().abs() @ s0[0, h].double().abs())
            both = o2[0, t - cut, h] if t >= cut else o1[0, t, h]
            for got in (o[0, t, h], both):
                _close(got, _np(want), _np(mag), 64 * dk + 1000, dtype, f"o at {t}")
        end = torch.exp((T - 1 - torch.arange(T, device="cuda", dtype=torch.float64)) * ld[h].double())[:, None]
        want = (K * end).T @ V + torch.exp(T * ld[h].double()) * s0[0, h].double()
        mag = (K * end).abs().T @ V.abs()
        for got in (s[0, h], s2[0, h]):
            # memories of at most ~1000 tokens: that many roundings of the state that still count
            _close(got, _np(want), _np(mag) + 1e-9, 4096, F32, "state")


def test_repeated_calls_give_the_same_bits():
    for dtype in (F32, BF16):
        a, n = _make(2, 3000, 4, 2, 64, 64, dtype)
        args = (a["q"], a["k"], a["v"], a["log_decay"])
        do = n(2, 3000, 4, 64)
        first = fw.linear_attention(*args, s0=a["s0"])
        grads = fw.linear_attention_backward(*args, do, s0=a["s0"])
        for _ in range(3):
            for x, y in zip(first, fw.linear_attention(*args, s0=a["s0"])):
                assert torch.equal(x, y)
            again = fw.linear_attention_backward(*args, do, s0=a["s0"])
            assert all(torch.equal(grads[n_], again[n_]) for n_ in grads)


def _check_backward(a, do, ds, lengths=None, scale=None):
    q, k, v, ld, s0 = (a[n] for n in ("q", "k", "v", "log_decay", "s0"))
    B, T, H, dk = q.shape
    Hkv, dv, sc = k.shape[2], v.shape[3], dk ** -0.5 if scale is None else scale
    got = fw.linear_attention_backward(q, k, v, ld, do, s0=s0, ds=ds, lengths=lengths, scale=scale)
    ln = None if lengths is None else lengths.tolist()
    arr = [_np(x) for x in (q, k, v, do)]
    if ln is not None:
        for x in arr:
            for b, L in enumerate(ln):
                x[b, L:] = 0
    q, k, v, do = arr
    s0, ds, ld = _np(s0), _np(ds), _np(ld)
    ab = lambda x: None if x is None else abs(x)
    want = oracle.backward(q, k, v, ld, do, s0, ds, ln, sc)
    mag = oracle.backward(ab(q), ab(k), ab(v), ld, ab(do), ab(s0), ab(ds), ln, abs(sc))
    n = dk + dv + T + 64 + H // Hkv
    for name, w, m in zip(("dq", "dk", "dv", "ds0"), want, mag):
        if got[name] is None:
            assert name == "ds0" and s0 is None
            continue
        _close(got[name], w, m, n, F32 if name == "ds0" else a["q"].dtype, name)
    if ln is not None:
        for b, L in enumerate(ln):
            assert not got["dq"][b, L:].any() and not got["dk"][b, L:].any() and not got["dv"][b, L:].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", SIZES)
def test_backward(size, dtype):
    B, T, H, Hkv, dk, dv = size
    a, n = _make(*size, dtype)
    _check_backward(a, n(B, T, H, dv), n(B, H, dk, dv, dt=F32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("start,last", [(False, False), (True, False), (False, True)])
def test_backward_without_states(dtype, start, last):
    a, n = _make(2, 333, 4, 2, 64, 96, dtype, start=start)
    _check_backward(a, n(2, 333, 4, 96), n(2, 4, 64, 96, dt=F32) if last else None, scale=0.25)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_backward_padded_batch_and_extreme_decays(dtype):
    T = 1100
    a, n = _make(4, T, 4, 1, 48, 64, dtype, decay=[0.0, -0.3, -50.0, float("-inf")])
    do = n(4, T, 4, 64)
    lengths = torch.tensor([T, 0, 1, 700], dtype=torch.int32, device="cuda")
    for b, L in enumerate(lengths.tolist()):
        for x in (a["q"], a["k"], a["v"], do):
            x[b, L:] = float("nan")
    _check_backward(a, do, n(4, 4, 48, 64, dt=F32), lengths)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(32, 65), (31, 96), (64, 90), (96, 66), (95, 96), (96, 97), (97, 96), (128, 95),
                                   (72, 72), (8, 94)])
def test_widths_around_a_tile(dk, dv, dtype):
    """Widths on both sides of 64 and 96, whole and odd: which columns a block takes, and which it has no more."""
    B, T, H, Hkv = 2, 201, 2, 1
    a, n = _make(B, T, H, Hkv, dk, dv, dtype)
    lengths = torch.tensor([T, 97], dtype=torch.int32, device="cuda")
    _check_forward(a)
    _check_forward(a, lengths=lengths)
    _check_backward(a, n(B, T, H, dv), n(B, H, dk, dv, dt=F32), lengths)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [65, 127, 128, 191, 896, 1023, 1024, 1281, 2048, 2177])
def test_lengths_around_a_split(T, dtype):
    """Lengths on both sides of where time is split into segments, full ones and one that ends a token early."""
    B, H, Hkv, dk, dv = 2, 4, 2, 64, 64
    a, n = _make(B, T, H, Hkv, dk, dv, dtype)
    do, ds = n(B, T, H, dv), n(B, H, dk, dv, dt=F32)
    lengths = torch.tensor([T // 2, T - 1], dtype=torch.int32, device="cuda")
    _check_forward(a)
    _check_forward(a, lengths=lengths)
    _check_backward(a, do, ds)
    _check_backward(a, do, ds, lengths)


def test_backward_against_differences_of_the_forward():
    """Directional derivatives in fp32: the forward pass is bilinear in each operand, so a central difference with
    any step has no truncation error; its rounding is that of two forward passes, each within n 2^-24 of its sum
    over absolute values."""
    a, n = _make(2, 90, 4, 2, 32, 48, F32)
    B, T, H, dk, dv = 2, 90, 4, 32, 48
    do, ds = n(B, T, H, dv), n(B, H, dk, dv)
    got = fw.linear_attention_backward(a["q"], a["k"], a["v"], a["log_decay"], do, s0=a["s0"], ds=ds)

    def loss(**kw):
        x = {**a, **kw}
        o, s = fw.linear_attention(x["q"], x["k"], x["v"], a["log_decay"], s0=x["s0"])
        terms = torch.cat([(o * do).double().flatten(), (s * ds).double().flatten()])
        return float(terms.sum()), float(terms.abs().sum())

    for name, g in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("s0", "ds0")):
        d = torch.randn_like(a[name])
        (up, m1), (down, m2) = loss(**{name: a[name] + d}), loss(**{name: a[name] - d})
        want = float((got[g].double() * d.double()).sum())
        assert abs((up - down) / 2 - want) <= (dk + dv + T + 64) * 2.0 ** -24 * 8 * (m1 + m2), name


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,Hkv,dk,dv", [(1, 1, 1, 1, 1), (3, 4, 2, 64, 64), (2, 6, 1, 33, 5), (5, 2, 2, 128, 128),
                                           (1, 3, 3, 7, 127), (130, 2, 1, 16, 4)])
def test_step(B, H, Hkv, dk, dv, dtype):
    a, n = _make(B, 1, H, Hkv, dk, dv, dtype)
    q, k, v = a["q"][:, 0], a["k"][:, 0], a["v"][:, 0]
    state, ld = a["s0"], a["log_decay"]
    wo, ws = oracle.step(_np(q), _np(k), _np(v), _np(ld), _np(state), None, dk ** -0.5)
    mo, ms = oracle.step(abs(_np(q)), abs(_np(k)), abs(_np(v)), _np(ld), abs(_np(state)), None, dk ** -0.5)
    after = torch.full_like(state, float("nan"))
    o = fw.linear_attention_step(q, k, v, ld, state, out_state=after)
    # the step holds no bf16 rounding but the output's
    _close(o, wo, mo if dtype == F32 else 0 * mo + 2.0 ** -16 * dk * mo, dk + 16, dtype, "o")
    _close(after, ws, ms, dk + 16, F32, "state")
    o2 = fw.linear_attention_step(q, k, v, ld, state)  # in place
    assert torch.equal(o, o2) and torch.equal(after, state)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_step_slots(dtype):
    """A pool with spare slots, ended requests, slots out of range, and rows that share a slot (tokens in order)."""
    B, H, Hkv, dk, dv, n_slots = 9, 4, 2, 24, 40, 12
    a, n = _make(B, 1, H, Hkv, dk, dv, dtype)
    q, k, v, ld = a["q"][:, 0], a["k"][:, 0], a["v"][:, 0], a["log_decay"]
    pool = n(n_slots, H, dk, dv, dt=F32)
    slots = torch.tensor([3, -1, 7, 3, 0, 12, 11, 3, 7], dtype=torch.int32, device="cuda")
    wo, ws = oracle.step(_np(q), _np(k), _np(v), _np(ld), _np(pool), slots.tolist(), 0.5)
    mo, ms = oracle.step(abs(_np(q)), abs(_np(k)), abs(_np(v)), _np(ld), abs(_np(pool)), slots.tolist(), 0.5)
    before = pool.clone()
    other = torch.full_like(pool, 5.0)
    o = fw.linear_attention_step(q, k, v, ld, pool, slots=slots, scale=0.5, out_state=other)
    assert torch.equal(pool, before)
    used = sorted({s for s in slots.tolist() if 0 <= s < n_slots})
    free = [s for s in range(n_slots) if s not in used]
    assert bool((other[free] == 5.0).all())
    _close(o, wo, mo, dk + 16, dtype, "o")
    _close(other[used], ws[used], ms[used], dk + 16, F32, "state")
    assert not o[1].any() and not o[5].any()
    o2 = fw.linear_attention_step(q, k, v, ld, pool, slots=slots, scale=0.5)
    assert torch.equal(o, o2) and torch.equal(pool[used], other[used]) and torch.equal(pool[free], before[free])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_then_tokens_equals_whole_prompt(dtype):
    """As they are used in serving: a prompt in one call, its state handed to the single-token step."""
    T, P, H, Hkv, dk, dv = 140, 131, 4, 2, 64, 64
    a, _ = _make(3, T, H, Hkv, dk, dv, dtype, start=False)
    q, k, v, ld = (a[n] for n in ("q", "k", "v", "log_decay"))
    _, s = fw.linear_attention(q[:, :P], k[:, :P], v[:, :P], ld)
    rows = [fw.linear_attention_step(q[:, t], k[:, t], v[:, t], ld, s) for t in range(P, T)]
    wo, ws = oracle.forward(_np(q), _np(k), _np(v), _np(ld), None, None, dk ** -0.5)
    mo, ms = oracle.forward(abs(_np(q)), abs(_np(k)), abs(_np(v)), _np(ld), None, None, dk ** -0.5)
    _close(torch.stack(rows, 1), wo[:, P:], mo[:, P:], dk + dv + T + 64, dtype, "o")
    _close(s, ws, ms, dk + dv + T + 64, F32, "state")


def test_captured_calls_on_other_streams_and_memory():
    """Captured into a graph and replayed on new data; calls on two streams at once; an unaligned q."""
    dtype, B, T, H, dk, dv = BF16, 2, 700, 4, 64, 64
    a, n = _make(B, T, H, H, dk, dv, dtype)
    b, _ = _make(B, T, H, H, dk, dv, dtype, seed=9)
    do = n(B, T, H, dv)
    x = {m: a[m].clone() for m in a}
    call = lambda y: (fw.linear_attention(y["q"], y["k"], y["v"], y["log_decay"], s0=y["s0"]),
                      fw.linear_attention_backward(y["q"], y["k"], y["v"], y["log_decay"], do, s0=y["s0"], ds=y["s0"]))
    want_a, want_b = call(a), call(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (o, s), grads = call(x)
    for y, (want, wg) in ((b, want_b), (a, want_a)):
        for m in x:
            x[m].copy_(y[m])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(s, want[1])
        assert all(torch.equal(grads[m], wg[m]) for m in grads)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for i in range(6):
        y = (a, b)[i % 2]
        outs.append(fw.linear_attention(y["q"], y["k"], y["v"], y["log_decay"], s0=y["s0"], stream=streams[i % 2]))
    torch.cuda.synchronize()
    for i, (o, s) in enumerate(outs):
        want = (want_a, want_b)[i % 2][0]
        assert torch.equal(o, want[0]) and torch.equal(s, want[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_offsets_beyond_32_bits(dtype):
    """More than 2^31 elements in every operand: the last sequence's last tokens equal those of a call on a copy of
    them (the decay forgets everything before within 40 tokens, 2^-57), forward and backward."""
    torch.cuda.empty_cache()
    B, T, H, d, tail = 3, 70003, 84, 128, 256
    assert B * T * H * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(B, T, H, d, dtype=dtype, device="cuda").normal_(generator=g)
    ld = torch.full((H,), -1.0, device="cuda")
    end = x[2:, T - tail:].clone()
    o, s = fw.linear_attention(x, x, x, ld)
    oe, se = fw.linear_attention(end, end, end, ld)
    # both evaluate the same sums from another start: twice the tolerance of one (see above), magnitudes below 16 d
    step = 2.0 ** -7 if dtype == BF16 else 2.0 ** -15
    assert float((o[2:, T - tail + 64:].float() - oe[:, 64:].float()).abs().max()) <= 2 * step * 16 * d ** 0.5
    assert float((o[2:, T - tail + 64:].float() - oe[:, 64:].float()).norm() / oe[:, 64:].float().norm()) <= step
    assert float((s[2:] - se).norm() / se.norm()) <= 2.0 ** -15
    del o, s
    grads = fw.linear_attention_backward(x, x, x, ld, x)
    ge = fw.linear_attention_backward(end, end, end, ld, end)
    for n in ("dq", "dk", "dv"):
        a, b = grads[n][2:, T - tail + 64:].float(), ge[n][:, 64:].float()
        assert float((a - b).norm() / b.norm()) <= step, n
    del grads, x
    torch.cuda.empty_cache()


def test_step_offsets_beyond_32_bits():
    torch.cuda.empty_cache()
    n_slots, H, d = 33000, 4, 128
    pool = torch.zeros(n_slots, H, d, d, device="cuda")
    assert pool.numel() > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn(2, H, d, device="cuda", generator=g) for _ in range(3))
    ld = torch.zeros(H, device="cuda")
    slots = torch.tensor([n_slots - 1, 5], dtype=torch.int32, device="cuda")
    o = fw.linear_attention_step(q, k, v, ld, pool, slots=slots, scale=1.0)
    for b, i in enumerate(slots.tolist()):
        assert torch.equal(pool[i], k[b][:, :, None] * v[b][:, None, :])
        want = (q[b].double() * k[b].double()).sum(-1, keepdim=True) * v[b].double()
        mag = (q[b].double() * k[b].double()).abs().sum(-1, keepdim=True) * v[b].double().abs()
        assert bool(((o[b].double() - want).abs() <= (d + 4) * 2.0 ** -24 * mag).all())
    assert int((pool.view(n_slots, -1)[:, 0] != 0).sum()) == 2
    del pool
    torch.cuda.empty_cache()
