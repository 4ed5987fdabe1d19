"""The norm of a residual stream and its gradients in fp64 (numpy), with bounds on an fp32 evaluation."""
import numpy as np

from .bounds import U, Bound


def _on(x, lengths):
    if lengths is None:
        return np.ones(x.shape[:2] + (1,), bool)
    return (np.arange(x.shape[1])[None] < np.clip(np.asarray(lengths), 0, x.shape[1])[:, None])[..., None]


def forward(x, residual, weight, bias, rms, eps, lengths=None):
    """x [N, S, C] -> {y, r, stats: (value, bound)}."""
    on, C = _on(x, lengths), x.shape[-1]
    r = np.where(on, x, 0.0) + (0.0 if residual is None else np.where(on, residual, 0.0))
    er = np.zeros_like(r) if residual is None else U * np.abs(r)
    mean = np.zeros(r.shape[:2] + (1,)) if rms else r.mean(-1, keepdims=True)
    em = np.zeros_like(mean) if rms else er.mean(-1, keepdims=True) + (C + 2) * U * np.abs(r).mean(-1, keepdims=True)
    d, ed = r - mean, er + em + U * np.abs(r - mean)
    var = (d * d).mean(-1, keepdims=True) + eps
    evar = (2 * np.abs(d) * ed).mean(-1, keepdims=True) + (C + 4) * U * var
    # the mean's error does not move a variance about the mean to first order, but it does add its square
    evar = evar + em * em
    k = 1 / np.sqrt(var) if eps > 0 else 1 / np.sqrt(np.maximum(var, 1e-300))
    ek = k * (evar / (2 * var) + 4 * U)
    hat = Bound(d, ed) * Bound(k, ek)
    w = np.ones(C) if weight is None else weight
    b = np.zeros(C) if bias is None else bias
    y = Bound(hat.m, hat.e) * Bound(w) + Bound(b)
    return dict(y=(np.where(on, d * k * w + b, 0.0), y.e), r=(r, er),
                stats=(np.concatenate([mean, k], -1), np.concatenate([em, ek], -1)))


def backward(r, stats, dy, weight, dr, rms, lengths=None):
    """From given statistics; {dr, dweight, dbias: (value, bound)}."""
    on, C = _on(r, lengths), r.shape[-1]
    r, dy = np.where(on, r, 0.0), np.where(on, dy, 0.0)
    mean, k = np.where(on, stats[..., :1], 0.0), np.where(on, stats[..., 1:], 0.0)
    w = np.ones(C) if weight is None else weight
    d = Bound(r - mean, U * np.abs(r - mean))
    hat, bh = (r - mean) * k, d * Bound(k)
    u, bu = dy * w, Bound(dy) * Bound(w)
    mu, bmu = u.mean(-1, keepdims=True), bu.sum(-1)[..., None] * (1.0 / C)
    muh, bmuh = (u * hat).mean(-1, keepdims=True), (bu * bh).sum(-1)[..., None] * (1.0 / C)
    inner, binner = u - hat * muh, bu + bh * bmuh
    if not rms:
        inner, binner = inner - mu, binner + bmu
    g, bg = k * inner, Bound(k) * binner
    if dr is not None:
        dr = np.where(on, dr, 0.0)
        g, bg = g + dr, bg + Bound(dr)
    return dict(dr=(np.where(on, g, 0.0), bg.e), dweight=((dy * hat).sum((0, 1)), (Bound(dy) * bh).sum((0, 1)).e),
                dbias=(dy.sum((0, 1)), Bound(dy).sum((0, 1)).e))
