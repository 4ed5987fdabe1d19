"""Linear attention and group norm at the largest sizes that they take, and the kernel variants that only some widths
reach."""
import pytest
import torch

import newton_solve_nonlinear_b200 as fw
from oracle import linear_attention as oracle
from tests import test_gpu_layers_guard_bands as bands
from tests import test_gpu_linear_attention as attention
from tests.test_gpu_group_norm import _check, _make

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS24 = 2.0 ** -24


def _slices(n, step=1 << 27):
    return [slice(i, min(i + step, n)) for i in range(0, n, step)]


@pytest.mark.parametrize("behind", [0, 5])
def test_norm_of_the_longest_sequence(behind):
    """2^31 - 1 rows of one channel, all of them or all but the last five: every row is read and written once.

    A thread joins 8 of its rows at a time: 3.63e6 rows a block / 256 threads / 8 are 1772 joins in a row, and about 40
    more across the threads, the warps and the 592 blocks.  Each rounds the mean once and the squares four times, so the
    mean is within 1850 2^-24 (|mean| + the largest |x - mean|) and r within half of 4 * 1850 2^-24 of itself; y adds a
    bf16 rounding, 2^-8 |y|.  In the backward pass a sum holds 7085 additions a thread, 256 across the threads and 1184
    across the blocks: within 8600 2^-24 of the sum of absolute values."""
    torch.cuda.empty_cache()
    S = 2 ** 31 - 1
    L = S - behind
    x = torch.empty(1, S, 1, dtype=BF16, device="cuda").normal_(0.5, 1.5, generator=torch.Generator("cuda").manual_seed(1))
    x[0, L:] = float("nan")
    w, b = torch.tensor([1.25], device="cuda"), torch.tensor([0.75], device="cuda")
    lengths = torch.tensor([L], dtype=torch.int32, device="cuda") if behind else None
    y = torch.full_like(x, float("nan"))
    _, stats = fw.group_norm(x, 1, w, b, act="none", lengths=lengths, out=y)
    flat, out = x.view(-1), y.view(-1)
    total = sum(float(flat[s].sum(dtype=torch.float64)) for s in _slices(L))
    mean = total / L
    var = sum(float((flat[s].double() - mean).square().sum()) for s in _slices(L)) / L
    r = (var + 1e-5) ** -0.5
    most = max(float((flat[s].float() - mean).abs().max()) for s in _slices(L))
    tol_m, tol_r = 1850 * EPS24 * (abs(mean) + most), 2 * 1850 * EPS24
    assert abs(float(stats[0, 0, 0]) - mean) <= tol_m
    assert abs(float(stats[0, 0, 1]) - r) <= tol_r * r
    for s in _slices(L):
        hat = (flat[s].double() - mean) * r
        want = hat * 1.25 + 0.75
        tol = 1.25 * (r * tol_m + hat.abs() * tol_r) + 8 * EPS24 * (want.abs() + 2)
        assert bool(((out[s].double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all())
    assert not out[L:].any()
    del y, out
    g = fw.group_norm_backward(x, stats, x, 1, w, b, act="none", lengths=lengths)
    size = sum(float(flat[s].abs().sum(dtype=torch.float64)) for s in _slices(L))
    assert abs(float(g["dbias"]) - total) <= 8600 * EPS24 * size
    dx = g["dx"].view(-1)
    assert not dx[L:].any() and all(bool(torch.isfinite(dx[s]).all()) for s in _slices(L))
    # dx = r w (x - mean(x) - xhat mean(x xhat)) is zero here but for eps: |r w (x - mean)| eps r^2, and roundings
    for s in _slices(L):
        assert float(dx[s].float().abs().max()) <= 1.25 * r * most * (1e-5 * r * r + 4 * 8600 * EPS24)
    del x, g, dx, flat
    torch.cuda.empty_cache()


@pytest.mark.parametrize("act,gated", [("silu", False), ("none", True)])
def test_norm_of_more_statistics_than_the_join_has_blocks(act, gated):
    """N groups just above 2^20, each of two rows of one channel."""
    N, S, G = 1051, 2, 1000
    x, w, b, n = _make(N, S, G, F32)
    _check(x, G, w, b, gate=n(N, S, G) if gated else None, act=act, dy=n(N, S, G))


def test_norm_backward_of_more_statistics_than_a_grid_holds():
    """N groups = 2^31.  The last n's gradients equal those of a call on a copy of them, whose sums are the same ones;
    dbias is the sum of dy, 2^21 terms in 32 slices of 2^15 and two rows each: within 2^17 2^-24 of the sum of absolute
    values, and dweight, with terms dy xhat, |xhat| <= 1 within 2^-20, too."""
    torch.cuda.empty_cache()
    N, S, G = 2 ** 20, 2, 2048
    x = torch.empty(N, S, G, dtype=BF16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(2))
    w, b = torch.rand(G, device="cuda") + 0.5, torch.rand(G, device="cuda")
    y, stats = fw.group_norm(x, G, w, b, act="none")
    del y
    g = fw.group_norm_backward(x, stats, x, G, w, b, act="none")
    for at in (0, 2 ** 19 - 1, N - 3):
        part = slice(at, at + 3)
        e = fw.group_norm_backward(x[part].clone(), stats[part].clone(), x[part].clone(), G, w, b, act="none")
        assert torch.equal(g["dx"][part], e["dx"])
    total, size, hats = (torch.zeros(G, dtype=torch.float64, device="cuda") for _ in range(3))
    for i in range(0, N, 2 ** 15):
        d, st = x[i:i + 2 ** 15].double(), stats[i:i + 2 ** 15].double()
        total += d.sum((0, 1))
        size += d.abs().sum((0, 1))
        hats += (d * (d - st[:, None, :, 0]) * st[:, None, :, 1]).sum((0, 1))
    tol = 2.0 ** 17 * EPS24 * size
    assert bool(((g["dbias"] - total).abs() <= tol).all())
    assert bool(((g["dweight"] - hats).abs() <= tol).all())
    del x, stats, g
    torch.cuda.empty_cache()


# One row per statistic, by the vectors that a lane holds of a group: widths that are multiples of 4 but not of 8 from
# 132 to 1020 (8 vectors of 4), that are not multiples of 4 from 129 to 1023 (32 of 1), and multiples of 8 from 264 to
# 512 (2 of 8); few rows, and more than all CTAs take at once
WIDTHS = [(7, 3, 132), (5, 2, 1020), (4, 9, 516), (9, 3, 129), (3, 2, 1023), (6, 5, 386), (6, 2, 264), (4, 3, 512)]
MANY = [(5001, 3, 132), (2503, 2, 513), (3001, 2, 264)]
TYPES = [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)]


@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("N,G,cg", WIDTHS + MANY)
def test_norm_of_rows_with_several_vectors_a_lane(N, G, cg, dtype, out):
    x, w, b, n = _make(N, 1, G * cg, dtype)
    dy = n(N, 1, G * cg, dt=out)
    lengths = [i % 3 for i in range(N)]  # a third of the rows are empty
    _check(x, G, w, b, act="silu", out_dtype=out, dy=dy)
    _check(x, G, w, b, gate=n(N, 1, G * cg, dt=dtype), act="gelu", out_dtype=out, dy=dy, lengths=lengths)


@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("gated,ragged", [(False, False), (True, True)])
@pytest.mark.parametrize("N,G,cg", WIDTHS)
def test_norm_of_rows_between_guard_bands(N, G, cg, gated, ragged, dtype, out):
    bands.test_group_norm(N, 1, G, cg, gated, ragged, dtype, out)


@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("N,S,G,cg", [(256, 3, 2, 5), (257, 3, 2, 5), (700, 2, 4, 12), (1500, 7, 3, 16), (300, 1, 1, 1100)])
def test_norm_parameters_of_many_sequences(N, S, G, cg, dtype, out):
    """Up to 256 sequences the last launch sums the parameters' gradients, beyond them a launch of its own."""
    x, w, b, n = _make(N, S, G * cg, dtype)
    dy = n(N, S, G * cg, dt=out)
    _check(x, G, w, b, act="gelu", out_dtype=out, dy=dy)
    _check(x, G, w, b, gate=n(N, S, G * cg, dt=dtype), out_dtype=out, dy=dy, lengths=[i % (S + 1) for i in range(N)])


def test_norm_of_the_most_rows():
    """2^31 - 1 rows of one channel, each its own statistic: xhat is zero, so y is act(bias), and the mean is x itself."""
    torch.cuda.empty_cache()
    N = 2 ** 31 - 1
    x = torch.empty(N, 1, dtype=BF16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(3))
    w, b = torch.tensor([1.25], device="cuda"), torch.tensor([0.75], device="cuda")
    y, stats = fw.group_norm(x, 1, w, b, act="none")
    assert all(bool((y[s] == 0.75).all()) and bool((stats[s, 0, 0] == x[s, 0].float()).all()) for s in _slices(N))
    del y
    g = fw.group_norm_backward(x, stats, x, 1, w, b, act="none")
    total = sum(float(x[s].sum(dtype=torch.float64)) for s in _slices(N))
    size = sum(float(x[s].abs().sum(dtype=torch.float64)) for s in _slices(N))
    # 592 blocks of 256 rows in flight: 14170 terms a thread, 256 and 592 more across them
    assert abs(float(g["dbias"]) - total) <= 15100 * EPS24 * size
    assert float(g["dweight"]) == 0 and all(not bool(g["dx"][s].any()) for s in _slices(N))
    del x, stats, g
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_of_the_longest_sequence(dtype):
    """2^30 tokens.  The decay, e^-1 a token, forgets everything before within 40 tokens, 2^-57: the last tokens, and the
    first ones, equal those of calls on copies, whose sums start elsewhere.  In the 2-norm: fp32 results by 2^-15, far
    above their ~150 roundings of 2^-24; a bf16 result holds three roundings to bf16 (the weighted score, the state's copy,
    the output), each 2^-8 / sqrt(3) at most in the mean square, so two of them differ by less than 2^-8 sqrt(6 / 3) < 2^-7."""
    torch.cuda.empty_cache()
    T, d, tail = 2 ** 30, 8, 512
    x = torch.empty(1, T, 1, d, dtype=dtype, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(5))
    ld = torch.tensor([-1.0], device="cuda")
    rel = lambda a, b: float((a.float() - b.float()).norm() / b.float().norm())
    step = 2.0 ** -15 if dtype == F32 else 2.0 ** -7

    def same(a, b):
        assert rel(a, b) <= step

    end, start = x[:, -tail:].clone(), x[:, :tail].clone()
    o, s = fw.linear_attention(x, x, x, ld)
    oe, se = fw.linear_attention(end, end, end, ld)
    same(o[:, -tail + 64:], oe[:, 64:])
    assert rel(s, se) <= 2.0 ** -15
    same(o[:, :tail], fw.linear_attention(start, start, start, ld)[0])
    middle = slice(T // 2 - 300, T // 2 + 300)  # across a block of 2^29 tokens
    part = x[:, middle].clone()
    same(o[:, middle][:, 64:], fw.linear_attention(part, part, part, ld)[0][:, 64:])
    del o, s
    if dtype == BF16:
        g = fw.linear_attention_backward(x, x, x, ld, x)
        for at, keep in ((end, slice(64, tail)), (start, slice(0, tail - 64))):
            ge = fw.linear_attention_backward(at, at, at, ld, at)
            whole = slice(T - tail, T) if at is end else slice(0, tail)
            for name in ("dq", "dk", "dv"):
                same(g[name][:, whole][:, keep], ge[name][:, keep])
        del g
    del x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_of_the_most_sequences(dtype):
    """2^24 sequences of one token: o = scale (q . k) v and s = k v^T, in one chunk each."""
    torch.cuda.empty_cache()
    B, d = 2 ** 24, 8
    g = torch.Generator("cuda").manual_seed(6)
    q, k, v = (torch.empty(B, 1, 1, d, dtype=dtype, device="cuda").normal_(generator=g) for _ in range(3))
    ld = torch.tensor([-0.5], device="cuda")
    o, s = fw.linear_attention(q, k, v, ld, scale=1.0)
    dot = (q.float() * k.float()).sum(-1, keepdim=True)
    mag = (q.float() * k.float()).abs().sum(-1, keepdim=True) * v.float().abs()
    tol = (16 * EPS24 + (2.0 ** -8 if dtype == BF16 else 0)) * mag + (2.0 ** -8 * o.float().abs() if dtype == BF16 else 0)
    assert bool(((o.float() - dot * v.float()).abs() <= tol).all())
    assert torch.equal(s[:, 0], k[:, 0, 0, :, None].float() * v[:, 0, 0, None].float())
    after = torch.full_like(s, float("nan"))
    o1 = fw.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], ld, torch.zeros_like(s), scale=1.0, out_state=after)
    assert torch.equal(after, s)
    assert bool(((o1.float() - (dot * v.float())[:, 0]).abs() <= tol[:, 0]).all())
    del q, k, v, o, s, after, o1, mag, tol
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [70, 1300])
def test_attention_of_overlapping_and_shared_views(T, dtype):
    """Operands whose rows overlap (a window that moves by less than its width), are shared by all sequences, or are the
    same for all tokens: the results are those of copies."""
    B, H, d = 3, 4, 64
    g = torch.Generator("cuda").manual_seed(7)
    buf = torch.randn(B * 8 * T * H + 4096, device="cuda", generator=g).to(dtype)
    views = [buf.as_strided((B, T, H, d), (T * H * 8, H * 8, 8, 1)),  # a window that moves by 8
             buf.as_strided((B, T, H, d), (24, 16, 8, 1), 64),                # axes that run over the same elements
             buf[: T * H * 8 // 64 * 64].view(1, -1, 1, d)[:, :1].expand(B, T, H, d),
             buf.as_strided((1, T, H, d), (0, H * 8, 8, 1)).expand(B, T, H, d)]
    ld = torch.linspace(-0.01, -0.5, H, device="cuda")
    do = torch.randn(B, T, H, d, device="cuda", generator=g).to(dtype)
    for i, q in enumerate(views):
        k, v = views[(i + 1) % 4], views[(i + 2) % 4]
        c = [t.clone(memory_format=torch.contiguous_format) for t in (q, k, v)]
        for a, b in zip(fw.linear_attention(q, k, v, ld), fw.linear_attention(*c, ld)):
            assert torch.equal(a, b)
        one, two = fw.linear_attention_backward(q, k, v, ld, do), fw.linear_attention_backward(*c, ld, do)
        assert all(torch.equal(one[m], two[m]) for m in ("dq", "dk", "dv"))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_step_of_many_rows_of_one_slot(dtype):
    """All rows of a batch name one slot: they are a sequence, as the call over whole sequences has it."""
    B, H, d = 300, 2, 32
    g = torch.Generator("cuda").manual_seed(8)
    q, k, v = (torch.randn(B, H, d, device="cuda", generator=g).to(dtype) for _ in range(3))
    ld = torch.tensor([-0.01, -0.3], device="cuda")
    pool = torch.randn(5, H, d, d, device="cuda", generator=g)
    before = pool.clone()
    o = fw.linear_attention_step(q, k, v, ld, pool, slots=torch.full((B,), 3, dtype=torch.int32, device="cuda"))
    want, ws = oracle.forward(*(t[None].double().cpu().numpy() for t in (q, k, v)), ld.double().cpu().numpy(),
                              before[3:4].double().cpu().numpy(), None, d ** -0.5)
    mo, ms = oracle.forward(*(t[None].double().abs().cpu().numpy() for t in (q, k, v)), ld.double().cpu().numpy(),
                            before[3:4].double().abs().cpu().numpy(), None, d ** -0.5)
    n = d + B + 16  # roundings of a step's sums, and one a token of the state
    attention._close(o[None], want, mo if dtype == F32 else 0 * mo + 2.0 ** -15 * mo, n, dtype, "o")
    attention._close(pool[3:4], ws, ms, n, F32, "state")
    assert all(torch.equal(pool[i], before[i]) for i in (0, 1, 2, 4))
