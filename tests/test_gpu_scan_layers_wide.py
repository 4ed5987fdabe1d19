"""The kernels that the selective state space block takes for large calls, against 64 bits: scans that fill the card (four states
to a thread, no segments of time, several tiles to a group), steps whose lanes prepare each other's channels, convolutions
whose threads take several runs.  Bounds as in test_gpu_selective_scan.py, without an allowance for segments where time is not
split, and with that of the sums that are really made where it is."""
import numpy as np
import pytest
import torch

import newton_solve_nonlinear_b200 as fw
from newton_solve_nonlinear_b200 import binding
from oracle.selective_scan import Scan
from tests.test_gpu_causal_conv import _make as _make_conv
from tests.test_gpu_causal_conv import _run as _run_conv
from tests.test_gpu_selective_scan import BF16, F32, _close, _make, _np

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _segments(p, o):
    """How many segments of time the call takes, by its workspace."""
    ops = binding._scan_operands(*p.values(), *(o.get(k) for k in ("skip", "gate", "dt_bias")), o["softplus"])
    need = binding.lib().pararnn_selective_scan_workspace_size(ops[0])
    s = ops[0]
    return 1 if need == 1 else max(2, round(need / (4 * s.B * s.D * (s.N + 1))))


def _check(p, o, n, segments, lengths=None):
    """Forward and backward, with and without the kept states.  segments: 1, or more, as the size is meant to give.  A segment's
    sum of steps is a chain in each of two threads or more and a sum over those: a rounding for each two of its tokens, and 40."""
    made = _segments(p, o)
    assert (made == 1) == (segments == 1)
    T = p["x"].shape[1]
    joined = 0 if made == 1 else (T // (made - 1) + 16) // 2 + 40
    q = {k: _np(v) for k, v in p.items()}
    r = {k: _np(v) if torch.is_tensor(v) else v for k, v in o.items() if k != "softplus"}
    ln = None if lengths is None else lengths.tolist()
    oracle = Scan(*q.values(), use_softplus=o["softplus"], lengths=ln, joined=joined, **r)
    want = oracle.forward()
    y, h, kept = fw.selective_scan(*p.values(), lengths=lengths, keep=True, **o)
    _close(y, want["y"], "y")
    _close(h, want["h"], "h")
    value, bound = oracle.kept()
    for b in range(p["x"].shape[0]):
        k = ((T if ln is None else min(max(ln[b], 0), T)) + 7) // 8
        _close(kept[b, :k], (value[b, :k], bound[b, :k]), f"kept {b}")
    dy, dh = n(*p["x"].shape), n(*h.shape, dt=F32)
    g = fw.selective_scan_backward(*p.values(), dy, dh=dh, lengths=lengths, kept=kept, **o)
    again = fw.selective_scan_backward(*p.values(), dy, dh=dh, lengths=lengths, **o)
    for k, v in oracle.backward(_np(dy), _np(dh)).items():
        _close(g[k], v, k)
        assert (v is None and again[k] is None) or torch.equal(g[k], again[k]), k


# B, T, G, channels of a group, N: at least 100 CTAs of 256 / lanes channels each; a group of two tiles, of one whole tile, of one
# odd one; states that fill their lanes and that do not, with and without aligned quads
WIDE = [(10, 17, 5, 130, 8), (10, 9, 5, 129, 6), (10, 18, 5, 130, 3), (10, 17, 5, 130, 1), (5, 19, 10, 66, 16), (5, 16, 5, 256, 16),
        (5, 33, 10, 65, 16), (4, 17, 13, 66, 13), (4, 17, 13, 66, 12), (5, 17, 10, 34, 32), (5, 20, 10, 34, 30), (5, 9, 10, 33, 17),
        (5, 17, 10, 18, 64), (5, 15, 10, 17, 64), (5, 8, 10, 18, 35), (1, 100, 100, 2, 16), (1, 75, 100, 1, 64), (1, 300, 100, 1, 16)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", WIDE)
def test_scans_that_fill_the_card(size, dtype):
    p, o, n = _make(*size, dtype, seed=31)
    _check(p, o, n, 1)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [(10, 30, 5, 130, 8), (5, 30, 10, 66, 16), (5, 30, 10, 34, 32), (5, 30, 10, 18, 64)])
def test_padded_scans_that_fill_the_card(size, dtype):
    p, o, n = _make(*size, dtype, seed=32)
    lengths = [30, 0, 1, 16, 23, 29, 8, 17, -1, 40][:size[0]]
    for b, L in enumerate(lengths):
        for t in (p["x"], p["dt"], p["b"], p["c"], o["gate"]):
            t[b, min(max(L, 0), 30):] = float("nan")
    _check(p, o, n, 1, torch.tensor(lengths, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("rate,step", [(1e-3, 0.002), (1.0, 5.0)])
def test_slow_and_fast_decays_of_scans_that_fill_the_card(rate, step):
    p, o, n = _make(5, 200, 10, 66, 16, F32, rate=rate, step=step, seed=33)
    _check(p, o, n, 1)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [(1, 2000, 1, 20, 16), (2, 900, 1, 40, 64), (1, 3000, 2, 3, 5), (3, 700, 1, 200, 2), (5, 700, 2, 10, 12)])
def test_segments_to_the_digits_of_their_own_sums(size, dtype):
    p, o, n = _make(*size, dtype, seed=34)
    _check(p, o, n, 2)


def test_slow_decays_over_segments():
    """As above, with memories of 5e5 tokens: what the join adds to a decay counts whole."""
    p, o, n = _make(1, 4000, 1, 12, 16, F32, rate=1e-3, step=0.002, seed=35)
    _check(p, o, n, 2)


def _in_order(slots, n_slots):
    """Rows of each slot in row order, as sequences: (rows [n_slots, most], lengths)."""
    rows = [[i for i, s in enumerate(slots) if s == k] for k in range(n_slots)]
    most = max(1, max(map(len, rows)))
    return np.array([r + [0] * (most - len(r)) for r in rows]), [len(r) for r in rows]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,G,per,N", [(230, 4, 64, 16), (240, 1, 300, 16), (460, 1, 256, 8), (120, 8, 32, 32), (60, 2, 150, 64),
                                       (230, 64, 4, 16), (930, 3, 20, 12)])
def test_steps_of_more_than_888_ctas(B, G, per, N, dtype):
    """Lanes take two channels, in two groups where groups are narrow, and prepare one each.  Some slots repeat, up to five
    times, and some name no state: tokens of one slot follow each other, so they are a sequence to the oracle."""
    p, o, n = _make(B, 1, G, per, N, dtype, seed=36)
    q = {k: v[:, 0] if v.dim() > 2 else v for k, v in p.items()}
    m = {k: v[:, 0] if k == "gate" else v for k, v in o.items() if k != "h0"}
    D, pool = G * per, B + 9
    r = np.random.default_rng(B)
    slots = r.permutation(pool)[:B]
    slots[r.choice(B, 12, replace=False)] = [slots[0]] * 4 + [slots[1]] * 3 + [slots[B - 1], -1, pool, -5, 1 << 30]
    state = n(pool, D, N, dt=F32)
    before, after = state.clone(), torch.full_like(state, 7.0)
    ts = torch.tensor(slots, dtype=torch.int32, device="cuda")
    y = fw.selective_scan_step(*q.values(), state, slots=ts, out_state=after, **m)
    rows, lengths = _in_order(slots.tolist(), pool)
    seq = {k: _np(v) if k == "a" else _np(v)[rows] for k, v in q.items()}
    kw = {k: _np(v)[rows] if k == "gate" else _np(v) for k, v in m.items() if torch.is_tensor(v)}
    want = Scan(*seq.values(), use_softplus=True, h0=_np(before), lengths=lengths, joined=0, **kw).forward()
    assert torch.equal(state, before)
    value, bound = np.zeros((B, D)), np.zeros((B, D))
    for k, L in enumerate(lengths):
        value[rows[k, :L]], bound[rows[k, :L]] = want["y"][0][k, :L], want["y"][1][k, :L]
    _close(y, (value, bound), "y")
    used = np.array(lengths) > 0
    _close(after[torch.from_numpy(used).cuda()], (want["h"][0][used], want["h"][1][used]), "state")
    assert (after[torch.from_numpy(~used).cuda()] == 7.0).all()
    assert torch.equal(fw.selective_scan_step(*q.values(), state, slots=ts, **m), y)
    assert torch.equal(state[torch.from_numpy(used).cuda()], after[torch.from_numpy(used).cuda()])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,D,W", [(20, 21, 16384, 4), (17, 70, 9472, 3), (9, 13, 16385, 5), (25, 1, 16384, 8)])
def test_convolutions_of_several_runs_to_a_thread(B, T, D, W, dtype):
    """More sequences than a thread's row of the grid has places: a thread takes one after another."""
    p, state, n = _make_conv(B, T, D, W, dtype, seed=37)
    _run_conv(p, state, n, "silu")
    lengths = torch.tensor([(7 * b) % (T + 1) for b in range(B)], dtype=torch.int32, device="cuda")
    for b, L in enumerate(lengths.tolist()):
        p["x"][b, L:] = float("nan")
    _run_conv(p, state, n, "silu", lengths)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_taps_gradients_of_a_million_tokens(dtype):
    """Against 64 bits on the device: what fp32 makes of q = dy silu'(p) at each token (below), a rounding for its product with x,
    and of the sums' terms a thread's pieces of 64 tokens, the chain of them and 40 for the sums over threads and CTAs."""
    T, D, W = 1 << 20, 32, 4
    p, _, n = _make_conv(1, T, D, W, dtype, seed=38)
    dy = n(1, T, D)
    g = fw.causal_conv_backward(p["x"], p["weight"], dy, p["bias"])
    x, v, w = p["x"].double()[0], dy.double()[0], p["weight"].double()
    full = torch.cat([x.new_zeros(W - 1, D), x])
    pre = sum(w[:, j] * full[j:j + T] for j in range(W)) + p["bias"].double()
    size = sum((w[:, j] * full[j:j + T]).abs() for j in range(W)) + p["bias"].double().abs()
    s = torch.sigmoid(pre)
    q = v * s * (1 + pre * (1 - s))
    # the slope's derivative is at most 1/2: (W + 1) U of the size of p's sum, half of that; ten U of the sigmoid's own, times
    # 1 + |p|; four roundings
    eq = v.abs() * ((W + 1) * U * size + (14 * (1 + pre.abs()) * s + 4) * U)
    sums = 32 + T / 8192 + 40
    for j in range(W):
        term = q * full[j:j + T]
        tol = (eq * full[j:j + T].abs()).sum(0) + sums * U * term.abs().sum(0)
        assert bool(((g["dweight"][:, j].double() - term.sum(0)).abs() <= tol).all()), j
    assert bool(((g["dbias"].double() - q.sum(0)).abs() <= eq.sum(0) + sums * U * q.abs().sum(0)).all())
