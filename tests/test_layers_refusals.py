"""What linear attention and group norm refuse, on the host and before anything is enqueued.  CPU only."""
import ctypes

import pytest
import torch

from newton_solve_nonlinear_b200 import binding

F32, BF16 = binding.F32, binding.BF16


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(binding._LIB_PATH):
        from newton_solve_nonlinear_b200 import build
        build.build()
    return binding.lib()


def _shape(**kw):
    a = dict(B=2, T=100, H=4, Hkv=2, dk=64, dv=32, dtype=F32, scale=0.125)
    a.update(kw)
    return binding.AttentionShape(*(a[n] for n in ("B", "T", "H", "Hkv", "dk", "dv", "dtype", "scale")))


BAD_SHAPES = [dict(B=0), dict(T=0), dict(H=0), dict(Hkv=0), dict(Hkv=3), dict(H=2, Hkv=4), dict(dk=0), dict(dk=129),
              dict(dv=0), dict(dv=129), dict(dtype=2), dict(scale=float("nan")), dict(scale=float("inf")),
              dict(B=1 << 20, H=32, Hkv=32)]


# addresses that are only compared, never read: the calls below refuse before any launch
BASE = 1 << 40


def _rows(at, T=100, heads=4, width=64, **kw):
    a = dict(ptr=at, stride_b=T * heads * width, stride_t=heads * width, stride_h=width)
    a.update(kw)
    return binding.Rows(a["ptr"], a["stride_b"], a["stride_t"], a["stride_h"])


@pytest.mark.parametrize("bad", BAD_SHAPES)
def test_attention_shapes(L, bad):
    r = _rows(BASE)
    assert L.pararnn_linear_attention_workspace_size(_shape(), r, r, r) > 0
    assert L.pararnn_linear_attention_backward_workspace_size(_shape(), r, r, r, r) > 0
    assert L.pararnn_linear_attention_workspace_size(_shape(**bad), r, r, r) == 0
    assert L.pararnn_linear_attention_backward_workspace_size(_shape(**bad), r, r, r, r) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_longest_sequence(L, dtype):
    """Tokens are counted in 32 bits: up to 2^30 of them."""
    r = _rows(BASE, T=1 << 30, heads=1, width=8)
    shape = lambda t: _shape(B=1, T=t, H=1, Hkv=1, dk=8, dv=8, dtype=dtype)
    size = lambda t: L.pararnn_linear_attention_workspace_size(shape(t), r, r, r)
    back = lambda t: L.pararnn_linear_attention_backward_workspace_size(shape(t), r, r, r, r)
    assert size(1 << 30) > 1 and back(1 << 30) > 1
    for t in ((1 << 30) + 1, (1 << 31) - 100, (1 << 31) - 1):
        assert size(t) == 0 and back(t) == 0


def test_workspace_by_operands(L):
    """bf16 rows off 16 bytes, or shared by stride 0, are packed into the workspace; others are not."""
    s = _shape(dtype=BF16, H=4, Hkv=4, dv=64)
    r = lambda **kw: _rows(BASE, **kw)
    size = lambda *x: L.pararnn_linear_attention_workspace_size(s, *x)
    tensor = 2 * 100 * 4 * 64 * 2
    assert size(r(), r(), r()) == 1  # none
    for odd in (r(ptr=BASE + 2), r(stride_t=257), r(stride_h=0)):
        assert size(odd, r(), r()) == tensor
        assert size(odd, odd, odd) == 3 * tensor
    # fp32 needs none of it
    f = _shape(H=4, Hkv=4, dv=64)
    assert L.pararnn_linear_attention_workspace_size(f, r(ptr=BASE + 4), r(), r()) == 1
    # odd widths: the outputs leave through the workspace too
    s = _shape(dtype=BF16, H=4, Hkv=4, dv=63)
    assert size(r(), r(), r()) == tensor


def _attention(L, **kw):
    s = _shape(T=1000)  # few heads: split in time, so it needs a workspace
    good = [_rows(BASE, T=1000), _rows(2 * BASE, T=1000, heads=2), _rows(3 * BASE, T=1000, heads=2, width=32)]
    need = L.pararnn_linear_attention_workspace_size(s, *good)
    assert need > 256
    a = dict(q=good[0], k=good[1], v=good[2], ld=4 * BASE, s0=None,
             lengths=None, o=5 * BASE, s=6 * BASE, ws=7 * BASE, n=need)
    a.update(kw)
    return L.pararnn_linear_attention(s, a["q"], a["k"], a["v"], a["ld"], a["s0"], a["lengths"], a["o"], a["s"], a["ws"],
                                      a["n"], None)


def test_attention_arguments(L):
    invalid = 3
    for bad in (dict(q=_rows(None)), dict(k=_rows(2 * BASE + 1)), dict(v=_rows(3 * BASE, stride_t=-64)),
                dict(q=_rows(BASE, stride_h=-1)), dict(ld=None), dict(o=None), dict(s=None), dict(ws=None),
                dict(o=5 * BASE + 8), dict(s=6 * BASE + 4), dict(ws=7 * BASE + 128), dict(n=0), dict(s0=8 * BASE + 4),
                dict(lengths=8 * BASE + 2), dict(o=BASE), dict(o=2 * BASE + 16), dict(s=4 * BASE), dict(ws=5 * BASE),
                dict(s0=6 * BASE + 16), dict(lengths=5 * BASE + 4), dict(s=5 * BASE + 1024)):
        assert _attention(L, **bad) == invalid, bad
    assert L.pararnn_linear_attention(None, None, None, None, None, None, None, None, None, None, 0, None) == invalid


def test_attention_backward_arguments(L):
    s = _shape()
    need = L.pararnn_linear_attention_backward_workspace_size(s, _rows(BASE), _rows(2 * BASE, heads=2),
                                                              _rows(3 * BASE, heads=2, width=32), _rows(5 * BASE, width=32))

    def call(**kw):
        a = dict(q=_rows(BASE), k=_rows(2 * BASE, heads=2), v=_rows(3 * BASE, heads=2, width=32), ld=4 * BASE,
                 do=_rows(5 * BASE, width=32), s0=None, ds=None, ln=None, dq=6 * BASE, dk=7 * BASE, dv=8 * BASE, ds0=None,
                 ws=9 * BASE, n=need)
        a.update(kw)
        return L.pararnn_linear_attention_backward(s, a["q"], a["k"], a["v"], a["ld"], a["do"], a["s0"], a["ds"], a["ln"],
                                                   a["dq"], a["dk"], a["dv"], a["ds0"], a["ws"], a["n"], None)

    for bad in (dict(do=_rows(None)), dict(dq=None), dict(dk=None), dict(dv=None), dict(dq=BASE), dict(dk=6 * BASE),
                dict(dv=5 * BASE), dict(ds=10 * BASE, ds0=10 * BASE), dict(ds0=6 * BASE), dict(n=need - 1), dict(ws=1),
                dict(ds=10 * BASE + 4)):
        assert call(**bad) == 3, bad
    # where keys and values are shared the partial gradients of each head are kept in fp32
    assert need >= 2 * 100 * 4 * 64 * 4


def test_step_arguments(L):
    def call(s=None, **kw):
        s = s or _shape(T=1)
        a = dict(q=_rows(BASE, T=1), k=_rows(2 * BASE, T=1, heads=2), v=_rows(3 * BASE, T=1, heads=2, width=32),
                 ld=4 * BASE, state=5 * BASE, slots=None, n=2, o=6 * BASE, out=5 * BASE)
        a.update(kw)
        return L.pararnn_linear_attention_step(s, a["q"], a["k"], a["v"], a["ld"], a["state"], a["slots"], a["n"], a["o"],
                                               a["out"], None)

    for bad in (dict(s=_shape(T=2)), dict(s=_shape(T=1, dk=200)), dict(n=0), dict(n=3), dict(state=None), dict(out=None),
                dict(o=5 * BASE), dict(out=5 * BASE + 16), dict(state=5 * BASE + 4), dict(slots=7 * BASE + 1),
                dict(q=_rows(None)), dict(ld=None)):
        assert call(**bad) == 3, bad


def _norm(**kw):
    a = dict(N=3, S=10, C=64, groups=4, x_dtype=F32, y_dtype=BF16, act=1, eps=1e-5)
    a.update(kw)
    return binding.NormShape(*(a[n] for n in ("N", "S", "C", "groups", "x_dtype", "y_dtype", "act", "eps")))


@pytest.mark.parametrize("bad", [dict(N=0), dict(S=0), dict(C=0), dict(groups=0), dict(groups=5), dict(x_dtype=7),
                                 dict(y_dtype=-1), dict(act=3), dict(act=-1), dict(eps=-1.0), dict(eps=float("nan")),
                                 dict(C=4096, groups=4096), dict(N=1 << 20, S=1 << 12)])
def test_norm_shapes(L, bad):
    for size in (L.pararnn_group_norm_workspace_size, L.pararnn_group_norm_backward_workspace_size):
        assert size(_norm()) > 0 and size(_norm(S=1)) > 0
        assert size(_norm(**bad)) == 0


def test_norm_arguments(L):
    s = _norm()
    need, back = L.pararnn_group_norm_workspace_size(s), L.pararnn_group_norm_backward_workspace_size(s)

    def forward(**kw):
        a = dict(x=BASE, w=None, b=None, gate=None, ln=None, y=2 * BASE, st=3 * BASE, ws=4 * BASE, n=need)
        a.update(kw)
        return L.pararnn_group_norm(s, a["x"], a["w"], a["b"], a["gate"], a["ln"], a["y"], a["st"], a["ws"], a["n"], None)

    for bad in (dict(x=None), dict(y=None), dict(st=None), dict(ws=None), dict(x=BASE + 4), dict(w=BASE + 4),
                dict(y=BASE), dict(y=BASE + 64), dict(n=need - 1), dict(gate=2 * BASE), dict(st=2 * BASE), dict(ln=BASE + 1)):
        assert forward(**bad) == 3, bad

    def backward(**kw):
        a = dict(x=BASE, st=2 * BASE, dy=3 * BASE, w=None, b=None, gate=None, ln=None, dx=4 * BASE, dw=None, db=None,
                 dg=None, ws=5 * BASE, n=back)
        a.update(kw)
        return L.pararnn_group_norm_backward(s, a["x"], a["st"], a["dy"], a["w"], a["b"], a["gate"], a["ln"], a["dx"],
                                             a["dw"], a["db"], a["dg"], a["ws"], a["n"], None)

    for bad in (dict(dy=None), dict(dx=None), dict(st=None), dict(gate=6 * BASE), dict(dg=6 * BASE), dict(dx=3 * BASE),
                dict(dw=7 * BASE, db=7 * BASE), dict(n=back - 1), dict(dw=4 * BASE)):
        assert backward(**bad) == 3, bad


def test_binding_refuses_before_the_library():
    """Shapes, types and devices are checked in Python with an error that names the argument."""
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)
    ld = z(4)
    for q, k, v in ((z(2, 5, 4, 8), z(2, 5, 3, 8), z(2, 5, 3, 8)), (z(2, 5, 4, 200), z(2, 5, 4, 200), z(2, 5, 4, 8)),
                    (z(5, 4, 8), z(5, 4, 8), z(5, 4, 8)), (z(2, 0, 4, 8), z(2, 0, 4, 8), z(2, 0, 4, 8)),
                    (z(2, 5, 4, 8), z(2, 5, 4, 8), z(2, 5, 4, 8))):  # the last: not on a CUDA device
        with pytest.raises(ValueError):
            binding.linear_attention(q, k, v, ld)
    with pytest.raises(TypeError):
        binding.linear_attention(*(z(1, 2, 4, 8, dt=torch.float16) for _ in range(3)), ld)
    with pytest.raises(ValueError, match="gradient"):
        binding.linear_attention(*(z(1, 2, 4, 8) for _ in range(3)), ld.requires_grad_())
    with pytest.raises(ValueError):
        binding.linear_attention_step(z(2, 4, 8), z(2, 4, 8), z(2, 4, 8), z(4), z(2, 4, 8, 8))
    for x, g in ((z(4), 1), (z(0, 4), 1), (z(3, 6), 4), (z(3, 6), 0), (z(3, 6), 2)):
        with pytest.raises(ValueError):
            binding.group_norm(x, g)
    with pytest.raises(ValueError, match="act"):
        binding.group_norm(z(3, 6), 2, act="tanh")
    with pytest.raises(TypeError):
        binding.group_norm(z(3, 6, dt=torch.float64), 2)
