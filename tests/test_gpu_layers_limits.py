"""Linear attention and group norm at the largest sizes that they take, and the kernel variants that only some widths
reach."""
import pytest
import torch

import newton_solve_nonlinear_b200 as fw
from tests import test_gpu_layers_guard_bands as bands
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
