"""What the selective scan, the causal convolution and the stream's norm refuse, on the host and before anything is
enqueued, and the largest sizes they take.  CPU only."""
import pytest
import torch

from newton_solve_nonlinear_b200 import binding
from tests.test_layers_refusals import L  # noqa: F401 (a fixture)

F32, BF16 = binding.F32, binding.BF16
BASE = 1 << 40  # addresses that are only compared, never read: the calls below refuse before any launch
INVALID = 3


def _scan(**kw):
    a = dict(B=2, T=100, D=64, G=2, N=16, dtype=F32, softplus=1)
    a.update(kw)
    return binding.ScanShape(*a.values())


def _rows(at, T=100, width=64, heads=1, **kw):
    a = dict(ptr=at, stride_b=T * heads * width, stride_t=heads * width, stride_h=width)
    a.update(kw)
    return binding.Rows(*a.values())


def _conv(**kw):
    a = dict(B=2, T=100, D=64, W=4, dtype=F32, act=1)
    a.update(kw)
    return binding.ConvShape(*a.values())


def _stream(**kw):
    a = dict(N=2, S=100, C=64, x_dtype=BF16, r_dtype=F32, y_dtype=BF16, rms=0, eps=1e-5)
    a.update(kw)
    return binding.StreamShape(*a.values())


@pytest.mark.parametrize("bad", [dict(B=0), dict(T=0), dict(D=0), dict(G=0), dict(G=3), dict(N=0), dict(N=65), dict(dtype=2),
                                 dict(softplus=2), dict(T=(1 << 30) + 1), dict(B=1 << 20, D=1 << 12)])
def test_scan_shapes(L, bad):  # noqa: F811
    assert L.pararnn_selective_scan_workspace_size(_scan()) > 0
    assert L.pararnn_selective_scan_workspace_size(_scan(**bad)) == 0
    for kept in (0, 1):
        assert L.pararnn_selective_scan_backward_workspace_size(_scan(), kept) > 0
        assert L.pararnn_selective_scan_backward_workspace_size(_scan(**bad), kept) == 0


def test_scan_workspaces(L):  # noqa: F811
    """Few channels and many tokens are split in time; the states that are not given are formed in the workspace."""
    assert L.pararnn_selective_scan_workspace_size(_scan(B=64, D=8192, T=64)) == 1  # none
    assert L.pararnn_selective_scan_workspace_size(_scan(T=1 << 20, B=1)) > 64 * 16 * 4
    back = lambda k: L.pararnn_selective_scan_backward_workspace_size(_scan(B=4, D=4096, G=1), k)
    assert back(0) == back(1) + (4 * 13 * 4096 * 16 * 4 + 255) // 256 * 256
    assert L.pararnn_selective_scan_workspace_size(_scan(B=1, T=1 << 30, D=1, G=1, N=1)) > 0


@pytest.mark.parametrize("T", [1, 7, 8, 9, 1000])
def test_scan_arguments(L, T):  # noqa: F811
    s = _scan(T=T)
    need = L.pararnn_selective_scan_workspace_size(s)
    r = lambda k, **kw: _rows(k * BASE, T=T, **kw)
    bc = lambda k, **kw: _rows(k * BASE, T=T, heads=2, width=16, **kw)

    def call(**kw):
        a = dict(x=r(1), dt=r(2), a=3 * BASE, b=bc(4), c=bc(5), skip=None, gate=None, bias=None, h0=None, ln=None, y=6 * BASE,
                 h=7 * BASE, kept=None, ws=8 * BASE, n=need)
        a.update(kw)
        return L.pararnn_selective_scan(s, *a.values(), None)

    bad = [dict(x=_rows(None)), dict(dt=_rows(2 * BASE + 1)), dict(b=bc(4, stride_t=-1)), dict(c=_rows(None)), dict(a=None),
           dict(a=3 * BASE + 2), dict(y=None), dict(h=None), dict(y=6 * BASE + 8), dict(h=7 * BASE + 4), dict(kept=9 * BASE + 4),
           dict(gate=_rows(None)), dict(skip=9 * BASE + 1), dict(bias=9 * BASE + 2), dict(h0=9 * BASE + 8), dict(ln=9 * BASE + 2),
           dict(y=BASE), dict(h=3 * BASE), dict(kept=7 * BASE), dict(kept=2 * BASE + 16), dict(h0=7 * BASE + 16), dict(ln=6 * BASE),
           dict(gate=r(6)), dict(skip=7 * BASE)]
    if need > 1:
        bad += [dict(ws=None), dict(ws=8 * BASE + 16), dict(n=need - 1), dict(ws=6 * BASE)]
    for kw in bad:
        assert call(**kw) == INVALID, kw
    assert L.pararnn_selective_scan(None, *[None] * 14, 0, None) == INVALID


def test_scan_backward_arguments(L):  # noqa: F811
    s = _scan()
    n0, n1 = (L.pararnn_selective_scan_backward_workspace_size(s, k) for k in (0, 1))
    assert n0 > n1 > 256

    def call(**kw):
        a = dict(x=_rows(BASE), dt=_rows(2 * BASE), a=3 * BASE, b=_rows(4 * BASE, heads=2, width=16),
                 c=_rows(5 * BASE, heads=2, width=16), skip=None, gate=None, bias=None, dy=_rows(6 * BASE), h0=None, dh=None,
                 ln=None, kept=7 * BASE, dx=8 * BASE, ddt=9 * BASE, da=10 * BASE, db=11 * BASE, dc=12 * BASE, dskip=None,
                 dgate=None, dbias=None, dh0=None, ws=13 * BASE, n=n1)
        a.update(kw)
        return L.pararnn_selective_scan_backward(s, *a.values(), None)

    for kw in (dict(dy=_rows(None)), dict(kept=None), dict(dx=None), dict(ddt=None), dict(da=None), dict(db=None), dict(dc=None),
               dict(gate=_rows(14 * BASE)), dict(dgate=14 * BASE), dict(dx=BASE), dict(ddt=8 * BASE), dict(da=13 * BASE),
               dict(dskip=14 * BASE + 4), dict(dh=14 * BASE, dh0=14 * BASE), dict(h0=14 * BASE, dh0=14 * BASE), dict(kept=9 * BASE),
               dict(n=n1 - 1), dict(ws=13 * BASE + 8), dict(ws=None), dict(dbias=10 * BASE + 16), dict(kept=7 * BASE + 4)):
        assert call(**kw) == INVALID, kw


def test_step_arguments(L):  # noqa: F811
    s = _scan(T=1)
    z = lambda k, **kw: _rows(k * BASE, T=1, **kw)

    def call(shape=s, **kw):
        a = dict(x=z(1), dt=z(2), a=3 * BASE, b=z(4, heads=2, width=16), c=z(5, heads=2, width=16), skip=None, gate=None,
                 bias=None, state=6 * BASE, slots=None, n=2, y=7 * BASE, out=6 * BASE)
        a.update(kw)
        return L.pararnn_selective_scan_step(shape, *a.values(), None)

    for kw in (dict(shape=_scan(T=2)), dict(shape=_scan(T=1, N=65)), dict(n=0), dict(n=3), dict(state=None), dict(out=None),
               dict(y=None), dict(y=6 * BASE), dict(out=6 * BASE + 16), dict(state=6 * BASE + 4), dict(slots=8 * BASE + 1),
               dict(x=_rows(None)), dict(a=None), dict(y=BASE), dict(gate=_rows(None)), dict(slots=7 * BASE)):
        assert call(**kw) == INVALID, kw


@pytest.mark.parametrize("bad", [dict(B=0), dict(T=0), dict(D=0), dict(W=1), dict(W=9), dict(dtype=-1), dict(act=2), dict(act=-1),
                                 dict(T=(1 << 30) + 1), dict(B=1 << 20, D=1 << 12)])
def test_conv_shapes(L, bad):  # noqa: F811
    assert L.pararnn_causal_conv_backward_workspace_size(_conv()) > 0
    assert L.pararnn_causal_conv_backward_workspace_size(_conv(**bad)) == 0
    assert L.pararnn_causal_conv(_conv(**bad), _rows(BASE), 2 * BASE, None, None, None, 3 * BASE, 4 * BASE, None) == INVALID


def test_conv_arguments(L):  # noqa: F811
    s = _conv()

    def forward(**kw):
        a = dict(x=_rows(BASE), w=2 * BASE, b=None, state=None, ln=None, y=3 * BASE, last=4 * BASE)
        a.update(kw)
        return L.pararnn_causal_conv(s, *a.values(), None)

    for kw in (dict(x=_rows(None)), dict(w=None), dict(w=2 * BASE + 2), dict(b=5 * BASE + 1), dict(state=5 * BASE + 4), dict(y=None),
               dict(last=None), dict(y=3 * BASE + 4), dict(last=4 * BASE + 8), dict(y=BASE), dict(last=3 * BASE), dict(state=4 * BASE),
               dict(ln=5 * BASE + 1), dict(x=_rows(BASE, stride_b=-1)), dict(y=2 * BASE)):
        assert forward(**kw) == INVALID, kw
    need = L.pararnn_causal_conv_backward_workspace_size(s)

    def backward(**kw):
        a = dict(x=_rows(BASE), w=2 * BASE, b=None, dy=_rows(3 * BASE), state=None, dlast=None, ln=None, dx=4 * BASE, dw=5 * BASE,
                 db=None, ds=None, ws=6 * BASE, n=need)
        a.update(kw)
        return L.pararnn_causal_conv_backward(s, *a.values(), None)

    for kw in (dict(dy=_rows(None)), dict(dx=None), dict(dw=None), dict(ws=None), dict(n=need - 1), dict(ws=6 * BASE + 4),
               dict(dx=3 * BASE), dict(dw=4 * BASE), dict(db=5 * BASE), dict(ds=7 * BASE, dlast=7 * BASE), dict(ds=7 * BASE + 2),
               dict(dlast=7 * BASE + 2)):
        assert backward(**kw) == INVALID, kw

    def step(shape=_conv(T=1), **kw):
        a = dict(x=_rows(BASE, T=1), w=2 * BASE, b=None, state=3 * BASE, slots=None, n=2, y=4 * BASE, out=3 * BASE)
        a.update(kw)
        return L.pararnn_causal_conv_step(shape, *a.values(), None)

    for kw in (dict(shape=_conv(T=2)), dict(n=3), dict(n=0), dict(state=None), dict(out=None), dict(y=None), dict(y=3 * BASE),
               dict(out=3 * BASE + 16), dict(slots=5 * BASE + 2), dict(w=None), dict(x=_rows(None))):
        assert step(**kw) == INVALID, kw


@pytest.mark.parametrize("bad", [dict(N=0), dict(S=0), dict(C=0), dict(C=(1 << 30) + 1), dict(x_dtype=2), dict(r_dtype=-1),
                                 dict(y_dtype=3), dict(rms=2), dict(eps=-1.0), dict(eps=float("nan")), dict(N=1 << 20, S=1 << 12)])
def test_stream_shapes(L, bad):  # noqa: F811
    assert L.pararnn_layer_norm_backward_workspace_size(_stream()) > 0
    assert L.pararnn_layer_norm_backward_workspace_size(_stream(**bad)) == 0
    assert L.pararnn_layer_norm(_stream(**bad), BASE, None, None, None, None, 2 * BASE, None, 3 * BASE, None) == INVALID


def test_stream_arguments(L):  # noqa: F811
    s = _stream()

    def forward(**kw):
        a = dict(x=BASE, res=None, w=None, b=None, ln=None, y=2 * BASE, r=None, st=3 * BASE)
        a.update(kw)
        return L.pararnn_layer_norm(s, *a.values(), None)

    for kw in (dict(x=None), dict(y=None), dict(st=None), dict(res=4 * BASE), dict(r=4 * BASE), dict(x=BASE + 4), dict(y=BASE),
               dict(res=4 * BASE, r=4 * BASE + 16), dict(res=4 * BASE, r=2 * BASE), dict(w=5 * BASE + 4), dict(ln=5 * BASE + 1),
               dict(st=2 * BASE), dict(b=3 * BASE)):
        assert forward(**kw) == INVALID, kw
    need = L.pararnn_layer_norm_backward_workspace_size(s)

    def backward(**kw):
        a = dict(r=BASE, st=2 * BASE, dy=3 * BASE, w=None, dr_in=None, ln=None, dr=4 * BASE, dx=None, dw=None, db=None,
                 ws=5 * BASE, n=need)
        a.update(kw)
        return L.pararnn_layer_norm_backward(s, *a.values(), None)

    for kw in (dict(r=None), dict(st=None), dict(dy=None), dict(dr=None), dict(dr=BASE), dict(dx=4 * BASE), dict(dw=4 * BASE),
               dict(dw=6 * BASE, db=6 * BASE), dict(dr_in=4 * BASE + 16), dict(n=need - 1), dict(ws=None), dict(dx=6 * BASE + 2)):
        assert backward(**kw) == INVALID, kw


FAR = 2 ** 32 + 3  # what a 32-bit count would take for 3


def _far(*shape):
    return torch.zeros(*(1 for _ in shape)).expand(*shape)  # no memory behind it


def test_binding_refuses_before_the_library():
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)
    ok = dict(x=z(2, 5, 4), dt=z(2, 5, 4), a=z(4, 3), b=z(2, 5, 1, 3), c=z(2, 5, 1, 3))
    for kw in (dict(), dict(x=z(5, 4)), dict(b=z(2, 5, 3)), dict(a=z(4)), dict(b=z(2, 5, 3, 3), c=z(2, 5, 3, 3)),
               dict(b=z(2, 5, 1, 65), c=z(2, 5, 1, 65), a=z(4, 65)), dict(x=z(2, 0, 4)), dict(x=_far(FAR, 1, 4)),
               dict(x=_far(1, FAR, 4)), dict(x=_far(1, 1, FAR))):  # the first: not on a CUDA device
        with pytest.raises(ValueError):
            binding.selective_scan(**{**ok, **kw})
    with pytest.raises(TypeError):
        binding.selective_scan(**{**ok, "x": z(2, 5, 4, dt=torch.float16)})
    with pytest.raises(ValueError, match="no_grad"):
        binding.selective_scan(**{**ok, "a": z(4, 3).requires_grad_()})
    step = dict(x=z(2, 4), dt=z(2, 4), a=z(4, 3), b=z(2, 1, 3), c=z(2, 1, 3))
    for state in (z(2, 4, 3), z(3, 4, 3), z(2, 4), z(0, 4, 3), _far(FAR, 4, 3)):
        with pytest.raises(ValueError):
            binding.selective_scan_step(**step, state=state)
    for x, w in ((z(2, 5, 4), z(4, 4)), (z(2, 4), z(4, 4)), (z(2, 5, 4), z(4, 1)), (z(2, 5, 4), z(4, 9)), (z(2, 0, 4), z(4, 4)),
                 (_far(FAR, 1, 4), z(4, 4)), (_far(1, FAR, 4), z(4, 4))):
        with pytest.raises(ValueError):
            binding.causal_conv(x, w)
    with pytest.raises(ValueError, match="act"):
        binding.causal_conv(z(2, 5, 4), z(4, 4), act="gelu")
    with pytest.raises(ValueError, match="no_grad"):
        binding.causal_conv(z(2, 5, 4), z(4, 4).requires_grad_())
    for state in (z(2, 3, 4), z(3, 3, 4), z(2, 4)):
        with pytest.raises(ValueError):
            binding.causal_conv_step(z(2, 4), z(4, 4), state)
    for x in (z(4), z(0, 4), z(3, 4), _far(FAR, 4), _far(1, FAR, 4)):
        with pytest.raises(ValueError):
            binding.layer_norm(x)
    with pytest.raises(TypeError):
        binding.layer_norm(z(3, 4, dt=torch.float64))
    with pytest.raises(ValueError, match="no_grad"):
        binding.layer_norm(z(3, 4).requires_grad_())
    for r in (z(4), z(3, 4), _far(FAR, 4)):
        with pytest.raises(ValueError):
            binding.layer_norm_backward(r, z(3, 2), r)
