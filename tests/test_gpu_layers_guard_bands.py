"""Guard-band checks of linear attention and group norm: every operand, output and workspace sits between bands of
0xFF bytes (NaN as fp32 and bf16), outputs start as NaN and the workspace as 0xFF.  After the call the bands are
unchanged, no output holds a NaN, and the results are those of the same call on ordinary allocations, bit for bit
(these calls are deterministic).  The calls go through the C ABI, which takes every address from the caller."""
import pytest
import torch

import newton_solve_nonlinear_b200 as fw
from newton_solve_nonlinear_b200 import binding
from tests.test_gpu_guard_bands import Guarded

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _inputs(**shapes):
    g = torch.Generator(device="cuda").manual_seed(7)
    return {k: Guarded(s, dt, init=torch.randn(*s, device="cuda", generator=g).to(dt)) for k, (s, dt) in shapes.items()}


def _done(outs, others):
    torch.cuda.synchronize()
    for name, (got, want) in outs.items():
        assert bool(torch.isfinite(got.t.float()).all()), name
        assert torch.equal(got.t, want), name
    for g in (*others, *(got for got, _ in outs.values())):
        assert g.bands_intact()


def _ws(n):
    return Guarded((n,), torch.uint8)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("B,T,H,Hkv,dk,dv", [(1, 1, 1, 1, 1, 1), (2, 65, 4, 2, 64, 64), (2, 257, 2, 2, 33, 127),
                                             (3, 333, 4, 1, 128, 96), (1, 1000, 3, 3, 48, 100), (2, 129, 2, 1, 120, 8)])
def test_linear_attention(B, T, H, Hkv, dk, dv, ragged, dtype):
    L = binding.lib()
    st = (B, H, dk, dv)
    x = _inputs(q=((B, T, H, dk), dtype), k=((B, T, Hkv, dk), dtype), v=((B, T, Hkv, dv), dtype), do=((B, T, H, dv), dtype),
                s0=(st, F32), ds=(st, F32))
    ld = Guarded((H,), F32, init=torch.linspace(-0.02, -0.7, H, device="cuda"))
    ln = Guarded((B,), torch.int32, init=torch.tensor([max(T - 3 * b, 0) for b in range(B)], device="cuda")) if ragged else None
    lens = None if ln is None else ln.t
    shape, rq, rk, rv = binding._attention_shape(x["q"].t, x["k"].t, x["v"].t, ld.t, None)
    rdo = binding._rows(x["do"].t, "do", x["q"].t, (B, T, H, dv))
    p = lambda g: None if g is None else g.t.data_ptr()

    o, s = Guarded((B, T, H, dv), dtype), Guarded(st, F32)
    ws = _ws(L.pararnn_linear_attention_workspace_size(shape, rq, rk, rv))
    assert L.pararnn_linear_attention(shape, rq, rk, rv, p(ld), p(x["s0"]), p(ln), p(o), p(s), p(ws), ws.n, _stream()) == 0
    plain = {k: g.t.clone() for k, g in x.items()}
    a = (plain["q"], plain["k"], plain["v"], ld.t.clone())
    wo, wsn = fw.linear_attention(*a, s0=plain["s0"], lengths=lens)
    _done(dict(o=(o, wo), s=(s, wsn)), [ws, ld, *x.values()])

    g = dict(dq=Guarded((B, T, H, dk), dtype), dk=Guarded((B, T, Hkv, dk), dtype), dv=Guarded((B, T, Hkv, dv), dtype),
             ds0=Guarded(st, F32))
    ws = _ws(L.pararnn_linear_attention_backward_workspace_size(shape, rq, rk, rv, rdo))
    assert L.pararnn_linear_attention_backward(shape, rq, rk, rv, p(ld), rdo, p(x["s0"]), p(x["ds"]), p(ln), p(g["dq"]),
                                               p(g["dk"]), p(g["dv"]), p(g["ds0"]), p(ws), ws.n, _stream()) == 0
    want = fw.linear_attention_backward(*a, plain["do"], s0=plain["s0"], ds=plain["ds"], lengths=lens)
    _done({n: (g[n], want[n]) for n in g}, [ws, ld, *x.values()])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("B,T,H,Hkv,dk,dv", [(2, 70, 2, 1, 96, 80), (1, 161, 3, 3, 31, 95), (2, 1100, 2, 2, 66, 65),
                                             (1, 1153, 4, 2, 64, 64)])
def test_linear_attention_in_wide_tiles_and_segments(B, T, H, Hkv, dk, dv, ragged, dtype):
    test_linear_attention(B, T, H, Hkv, dk, dv, ragged, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,Hkv,dk,dv", [(1, 1, 1, 1, 1), (3, 4, 2, 64, 64), (2, 3, 3, 33, 127), (5, 2, 1, 128, 100)])
def test_step(B, H, Hkv, dk, dv, dtype):
    L = binding.lib()
    x = _inputs(q=((B, H, dk), dtype), k=((B, Hkv, dk), dtype), v=((B, Hkv, dv), dtype), state=((B + 2, H, dk, dv), F32))
    ld = Guarded((H,), F32, init=torch.linspace(-0.02, -0.7, H, device="cuda"))
    slots = Guarded((B,), torch.int32, init=torch.arange(B, 0, -1, device="cuda"))
    shape, rq, rk, rv = binding._attention_shape(x["q"].t, x["k"].t, x["v"].t, ld.t, None, 3)
    plain = {k: g.t.clone() for k, g in x.items()}
    o = Guarded((B, H, dv), dtype)
    assert L.pararnn_linear_attention_step(shape, rq, rk, rv, ld.t.data_ptr(), x["state"].t.data_ptr(), slots.t.data_ptr(),
                                           B + 2, o.t.data_ptr(), x["state"].t.data_ptr(), _stream()) == 0
    want = fw.linear_attention_step(plain["q"], plain["k"], plain["v"], ld.t.clone(), plain["state"], slots=slots.t.clone())
    _done(dict(o=(o, want), state=(x["state"], plain["state"])), [ld, slots, *x.values()])


@pytest.mark.parametrize("dtype,out", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("gated,ragged", [(False, False), (True, True)])
@pytest.mark.parametrize("N,S,G,cg", [(1, 1, 1, 1), (37, 1, 4, 33), (5, 1, 16, 128), (3, 1, 2, 600), (2, 1, 1, 1100),
                                      (3, 65, 5, 12), (2, 257, 4, 16), (2, 100, 3, 7), (1, 333, 2, 300)])
def test_group_norm(N, S, G, cg, gated, ragged, dtype, out):
    L, C = binding.lib(), G * cg
    x = _inputs(x=((N, S, C), dtype), dy=((N, S, C), out), w=((C,), F32), b=((C,), F32),
                **(dict(gate=((N, S, C), dtype)) if gated else {}))
    ln = Guarded((N,), torch.int32, init=torch.tensor([max(S - 2 * n, 0) for n in range(N)], device="cuda")) if ragged else None
    shape = binding._norm_shape(x["x"].t, G, "silu", 1e-5, out)
    p = lambda g: None if g is None else g.t.data_ptr()
    y, stats = Guarded((N, S, C), out), Guarded((N, G, 2), F32)
    ws = _ws(L.pararnn_group_norm_workspace_size(shape))
    gate = x.get("gate")
    assert L.pararnn_group_norm(shape, p(x["x"]), p(x["w"]), p(x["b"]), p(gate), p(ln), p(y), p(stats), p(ws), ws.n,
                                _stream()) == 0
    c = {k: g.t.clone() for k, g in x.items()}
    lens = None if ln is None else ln.t
    wy, wst = fw.group_norm(c["x"], G, c["w"], c["b"], gate=c.get("gate"), lengths=lens, out_dtype=out)
    _done(dict(y=(y, wy), stats=(stats, wst)), [ws, *x.values()])

    g = dict(dx=Guarded((N, S, C), dtype), dweight=Guarded((C,), F32), dbias=Guarded((C,), F32))
    if gated:
        g["dgate"] = Guarded((N, S, C), dtype)
    ws = _ws(L.pararnn_group_norm_backward_workspace_size(shape))
    assert L.pararnn_group_norm_backward(shape, p(x["x"]), p(stats), p(x["dy"]), p(x["w"]), p(x["b"]), p(gate), p(ln),
                                         p(g["dx"]), p(g["dweight"]), p(g["dbias"]), p(g.get("dgate")), p(ws), ws.n,
                                         _stream()) == 0
    want = fw.group_norm_backward(c["x"], wst, c["dy"], G, c["w"], c["b"], gate=c.get("gate"), lengths=lens)
    _done({n: (g[n], want[n]) for n in g}, [ws, *x.values()])
