"""The residual stream's norm on the GPU against fp64 and its running error bounds (oracle/layer_norm.py): elementwise what
fp32 may be off, and for results in bf16 half a step of 2^-8 of the value on top."""
import pytest
import torch

import newton_solve_nonlinear_b200 as fw
from oracle import layer_norm as oracle
from tests.test_gpu_selective_scan import BF16, F32, _close, _np

pytestmark = pytest.mark.gpu

TYPES = [(F32, F32, F32), (BF16, F32, BF16), (BF16, BF16, BF16), (F32, BF16, BF16), (BF16, BF16, F32)]


def _make(N, S, C, x, r, y, seed=0, mean=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, dt=F32: torch.randn(*s, device="cuda", generator=g).to(dt)
    return dict(x=n(N, S, C, dt=x), residual=(2 * n(N, S, C) + mean).to(r), weight=1 + 0.3 * n(C), bias=n(C)), n


def _run(p, n, y_dtype, rms, lengths=None, add=True, eps=1e-5):
    x, res, w, b = p["x"], p["residual"] if add else None, p["weight"], p["bias"]
    y, r, stats = fw.layer_norm(x, w, b, residual=res, rms=rms, eps=eps, lengths=lengths, out_dtype=y_dtype)
    ln = None if lengths is None else lengths.tolist()
    want = oracle.forward(_np(x), _np(res), _np(w), _np(b), rms, eps, ln)
    _close(y, want["y"], "y")
    _close(stats, want["stats"], "stats")
    if add:
        _close(r, want["r"], "r")
    else:
        assert r is x
    dy, dr = n(*x.shape, dt=y_dtype), n(*x.shape, dt=r.dtype) if add else None
    if ln is not None:
        for i, L in enumerate(ln):
            dy[i, max(L, 0):] = float("nan")
            if add:
                dr[i, max(L, 0):] = float("nan")
    g = fw.layer_norm_backward(r, stats, dy, w, b, dr=dr, rms=rms, lengths=lengths, dx_dtype=x.dtype)
    back = oracle.backward(_np(r), _np(stats), _np(dy), _np(w), _np(dr), rms, ln)
    for k in ("dr", "dweight", "dbias"):
        _close(g[k], back[k], k)
    _close(g["dx"], back["dr"], "dx")
    assert (g["dx"] is g["dr"]) == (x.dtype == r.dtype)
    return y, r, stats, g


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("N,S,C", [(1, 1, 1), (2, 3, 4), (1, 9, 5), (3, 1, 31), (1, 2, 128), (2, 5, 130), (1, 33, 256), (2, 2, 500),
                                   (1, 3, 512), (1, 2, 516), (2, 1, 1000), (1, 3, 1025), (1, 2, 2048), (1, 2, 2049), (1, 3, 4100),
                                   (1, 2, 8190), (1, 2, 8193), (1, 1, 10240), (1, 2, 32768), (1, 2, 32772), (1, 3, 9001)])
def test_sizes(N, S, C, rms, types):
    p, n = _make(N, S, C, *types)
    _run(p, n, types[2], rms)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("rows,C", [(5000, 64), (3000, 300), (700, 1028), (400, 9001)])
def test_many_rows(rows, C, rms):
    p, n = _make(2, rows // 2, C, BF16, F32, BF16, seed=1)
    _run(p, n, BF16, rms)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("C", [24, 700, 33000])
def test_without_a_residual(C, rms, types):
    p, n = _make(2, 3, C, types[0], types[0], types[2], seed=2)
    _run(p, n, types[2], rms, add=False)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("C", [24, 33, 1100, 33000])
def test_padded_batch(C, add, rms):
    p, n = _make(5, 7, C, BF16, F32 if add else BF16, BF16, seed=3)
    ln = torch.tensor([7, 0, -2, 3, 9], dtype=torch.int32, device="cuda")
    for i, L in enumerate(ln.clamp(0, 7).tolist()):
        p["x"][i, L:] = float("nan")
        p["residual"][i, L:] = float("inf")
    y, r, stats, g = _run(p, n, BF16, rms, ln.clamp(0, 7), add=add)
    raw = fw.layer_norm(p["x"], p["weight"], p["bias"], residual=p["residual"] if add else None, rms=rms, lengths=ln)
    assert torch.equal(raw[0], y) and torch.equal(raw[2], stats)
    for i, L in enumerate(ln.clamp(0, 7).tolist()):
        assert not y[i, L:].any() and not g["dr"][i, L:].any() and not g["dx"][i, L:].any()
        assert not add or not r[i, L:].any()


def test_large_common_offset():
    """Squares about the mean: an offset of 1000 with a spread of 2 costs fp32's own digits of r alone."""
    p, n = _make(1, 6, 2048, F32, F32, F32, seed=4, mean=1000.0)
    _run(p, n, F32, False)


def test_without_weight_and_bias_and_other_eps():
    p, n = _make(2, 3, 100, F32, F32, F32, seed=5)
    x, res = p["x"], p["residual"]
    y, r, stats = fw.layer_norm(x, residual=res, eps=0.1)
    want = oracle.forward(_np(x), _np(res), None, None, False, 0.1)
    _close(y, want["y"], "y")
    g = fw.layer_norm_backward(r, stats, y)
    _close(g["dr"], oracle.backward(_np(r), _np(stats), _np(y), None, None, False)["dr"], "dr")
    assert g["dweight"] is None and g["dbias"] is None
    flat = fw.layer_norm(x.reshape(6, 100), residual=res.reshape(6, 100), eps=0.1)
    assert torch.equal(flat[0], y.reshape(6, 100)) and flat[2].shape == (6, 2)


def test_in_place_repeated_and_in_a_graph():
    p, n = _make(2, 50, 768, BF16, F32, BF16, seed=6)
    dy, dr = n(2, 50, 768, dt=BF16), n(2, 50, 768)

    def run(**k):
        y, r, stats = fw.layer_norm(p["x"], p["weight"], p["bias"], residual=p["residual"])
        return y, r, stats, *fw.layer_norm_backward(r, stats, dy, p["weight"], p["bias"], dr=dr, dx_dtype=BF16, **k).values()

    first = run()
    for fill in (0x00, 0xFF):
        for u, v in zip(run(workspace=torch.full((1 << 22,), fill, dtype=torch.uint8, device="cuda")), first):
            assert torch.equal(u, v)
    stream, y = p["residual"].clone(), torch.empty_like(first[0])
    out = fw.layer_norm(p["x"], p["weight"], p["bias"], residual=stream, out=(y, stream))
    assert out[1] is stream and torch.equal(stream, first[1]) and torch.equal(y, first[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    p["x"].copy_(n(2, 50, 768)), dy.copy_(n(2, 50, 768))
    graph.replay()
    torch.cuda.synchronize()
    for u, v in zip(out, run()):
        assert torch.equal(u, v)


def test_refusals():
    p, n = _make(2, 3, 8, F32, F32, F32, seed=7)
    for kw in (dict(residual=p["residual"][:1]), dict(weight=p["weight"][:4]), dict(lengths=torch.zeros(2, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            fw.layer_norm(p["x"], **kw)
    with pytest.raises(ValueError):
        fw.layer_norm(p["x"].transpose(0, 1))
    with pytest.raises(ValueError):
        fw.layer_norm(p["x"], out=(torch.empty_like(p["x"]), torch.empty_like(p["x"])))
    y, r, stats = fw.layer_norm(p["x"], p["weight"])
    with pytest.raises(ValueError):
        fw.layer_norm_backward(r, stats[:1], y)
