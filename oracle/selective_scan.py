"""The selective state space scan and its gradients, token by token in fp64 (numpy), and bounds on an fp32 evaluation.

The core runs on plain arrays and on ``bounds.Bound`` alike.  Shapes: x, dt, gate [B, T, D]; b, c [B, T, G, N]; a [D, N]."""
import numpy as np

from . import bounds
from .bounds import U, Bound


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def _on(lengths, B, T):
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)
    return np.arange(T)[None] < n[:, None]


def _clean(x, on):
    return None if x is None else np.where(on.reshape(on.shape + (1,) * (x.ndim - 2)), x, 0.0)


def _forward(s, x, decay, b, c, skip, h0):
    """Inner outputs (before the gate) and the states, the one before the first token in front; b and c per channel."""
    h, hs, ys, u = h0, [h0], [], s * x
    for t in range(x.m.shape[1] if isinstance(x, Bound) else x.shape[1]):
        h = decay[:, t] * h + u[:, t][..., None] * b[:, t]
        hs.append(h)
        ys.append((c[:, t] * h).sum(-1) + skip * x[:, t])
    return bounds.stack(ys, 1), hs


def _backward(s, x, decay, a, b, c, skip, hs, v, dh):
    T = len(hs) - 1
    p, out = dh, {n: [None] * T for n in ("dx", "ds", "db", "dc")}
    da = None
    u = s * x
    for t in reversed(range(T)):
        g = p + v[:, t][..., None] * c[:, t]
        out["dc"][t] = v[:, t][..., None] * hs[t + 1]
        out["db"][t] = g * u[:, t][..., None]
        gb = (g * b[:, t]).sum(-1)
        out["dx"][t] = s[:, t] * gb + skip * v[:, t]
        p = decay[:, t] * g
        moved = p * hs[t]
        out["ds"][t] = (moved * a).sum(-1) + gb * x[:, t]
        add = (moved * s[:, t][..., None]).sum(0)
        da = add if da is None else da + add
    out = {n: bounds.stack(xs, 1) for n, xs in out.items()}
    return dict(out, da=da, dh0=p, dskip=(v * x).sum((0, 1)))


def _per_group(x, G):
    m = x.m if isinstance(x, Bound) else x
    B, T, D, N = m.shape
    return x.reshape(B, T, G, D // G, N).sum(3)


class Scan:
    """One call's operands; ``forward`` and ``backward`` give {name: (value, bound on fp32's error)}."""

    def __init__(self, x, dt, a, b, c, skip=None, gate=None, dt_bias=None, use_softplus=True, h0=None, lengths=None,
                 joined=None):
        """joined: of how many terms the sums of steps are that join segments of time; as many as there are tokens if None, 0
        where time is not split."""
        B, T, D = x.shape
        self.G, N = b.shape[2:]
        self.on = on = _on(lengths, B, T)
        self.given = dict(skip=skip is not None, gate=gate is not None, dt_bias=dt_bias is not None, h0=h0 is not None)
        self.x, dt, self.gate = _clean(x, on), _clean(dt, on), _clean(gate, on)
        rep = lambda m: np.repeat(_clean(m, on), D // self.G, axis=2)
        self.b, self.c, self.a = rep(b), rep(c), a
        self.skip = np.zeros(D) if skip is None else skip
        self.h0 = np.zeros((B, D, N)) if h0 is None else h0
        self.raw = dt + (0.0 if dt_bias is None else dt_bias)
        self.soft = use_softplus
        self.s = np.where(on[..., None], softplus(self.raw) if use_softplus else self.raw, 0.0)
        z = self.s[..., None] * a
        self.decay = np.exp(z)
        # what fp32 makes of the step: the sum rounds, softplus is within eight steps
        es = U * (np.abs(self.raw) * bounds.sigmoid(self.raw) + 16 * self.s) if use_softplus else U * np.abs(self.s)
        es = np.where(on[..., None], es, 0.0)
        # z's error: the step's, two roundings, and those of a sum of steps where segments join
        ez = es[..., None] * np.abs(a) + (2 + (T if joined is None else joined)) * U * np.abs(z)
        # a slow decay enters as exp(z) - 1, from its series, and as a product beside the old value, whose sum with the input
        # rounds once more; any other as exp(z) from ex2, within 1.3e-7 of itself.  (Above 0.01: a kernel may take the
        # difference a little further.)
        ed = self.decay * ez + np.where(np.abs(z) < 0.01, 8 * U * np.abs(np.expm1(z)) + 2 * U, 4 * U * self.decay)
        self.bs, self.bdecay = Bound(self.s, es), Bound(self.decay, np.where(on[..., None, None], ed, 0.0))

    def _bounds(self):
        return [Bound(v) for v in (self.x, self.b, self.c, self.skip, self.h0)]

    def forward(self):
        y, self.hs = _forward(self.s, self.x, self.decay, self.b, self.c, self.skip, self.h0)
        bx, bb, bc, bskip, bh0 = self._bounds()
        by, self.bhs = _forward(self.bs, bx, self.bdecay, bb, bc, bskip, bh0)
        self.inner, self.binner = y, by
        if self.gate is not None:
            y = y * (self.gate * bounds.sigmoid(self.gate))
            by = by * (Bound(self.gate) * bounds.sigmoid_bound(self.gate))
        y = np.where(self.on[..., None], y, 0.0)
        return dict(y=(y, by.e), h=(self.hs[-1], self.bhs[-1].e))

    def kept(self):
        """The states before every eighth token, and their bounds: [B, ceil(T / 8), D, N]."""
        every = range(0, len(self.hs) - 1, 8)
        return np.stack([self.hs[t] for t in every], 1), np.stack([self.bhs[t].e for t in every], 1)

    def backward(self, dy, dh=None):
        if not hasattr(self, "hs"):
            self.forward()
        dy = _clean(dy, self.on)
        dh = np.zeros_like(self.h0) if dh is None else dh
        v, bv = dy, Bound(dy)
        if self.gate is not None:
            v = dy * (self.gate * bounds.sigmoid(self.gate))
            bv = bv * (Bound(self.gate) * bounds.sigmoid_bound(self.gate))
        g = _backward(self.s, self.x, self.decay, self.a, self.b, self.c, self.skip, self.hs, v, dh)
        bx, bb, bc, bskip, _ = self._bounds()
        # the states that the backward pass forms again start from kept ones, so their bound is the forward's
        e = _backward(self.bs, bx, self.bdecay, Bound(self.a, 2 * U * np.abs(self.a)), bb, bc, bskip, self.bhs, bv, Bound(dh))
        ddt, bddt = g["ds"], e["ds"]
        if self.soft:
            ddt = ddt * bounds.sigmoid(self.raw)
            bddt = bddt * bounds.sigmoid_bound(self.raw, U * np.abs(self.raw))
        on = self.on[..., None]
        ddt, bddt = np.where(on, ddt, 0.0), Bound(bddt.m * on, bddt.e * on)
        out = dict(dx=(np.where(on, g["dx"], 0.0), e["dx"].e), ddt=(ddt, bddt.e), da=(g["da"], e["da"].e),
                   db=(_per_group(g["db"], self.G), _per_group(e["db"], self.G).e),
                   dc=(_per_group(g["dc"], self.G), _per_group(e["dc"], self.G).e), dskip=(g["dskip"], e["dskip"].e),
                   ddt_bias=(ddt.sum((0, 1)), bddt.sum((0, 1)).e), dh0=(g["dh0"], e["dh0"].e), dgate=None)
        if self.gate is not None:
            out["dgate"] = (np.where(on, dy * self.inner * bounds.silu_slope(self.gate), 0.0),
                            (Bound(dy) * self.binner * bounds.silu_slope_bound(self.gate)).e)
        for n, used in (("dskip", "skip"), ("ddt_bias", "dt_bias"), ("dh0", "h0")):
            if not self.given[used]:
                out[n] = None
        return out
