"""The short causal convolution over time and its gradients in fp64 (numpy), with bounds on an fp32 evaluation."""
import numpy as np

from . import bounds
from .bounds import Bound


def _inputs(x, state, W, lengths):
    B, T, D = x.shape
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)
    on = np.arange(T)[None] < n[:, None]
    first = np.zeros((B, W - 1, D)) if state is None else state
    return np.concatenate([first, np.where(on[..., None], x, 0.0)], 1), on, n


def _pre(full, weight, bias, T):
    W = weight.shape[1]
    value = sum(weight[:, j] * full[:, j:j + T] for j in range(W)) + bias
    size = sum((Bound(weight[:, j]) * Bound(full[:, j:j + T]) for j in range(W)), Bound(bias))
    return value, size


def forward(x, weight, bias, act, state=None, lengths=None):
    """{y: (value, bound), last: (value, 0)}."""
    T, W = x.shape[1], weight.shape[1]
    bias = np.zeros(x.shape[2]) if bias is None else bias
    full, on, n = _inputs(x, state, W, lengths)
    p, size = _pre(full, weight, bias, T)
    y, e = p, size.e
    if act == "silu":
        y = p * bounds.sigmoid(p)
        e = (Bound(p, size.e) * bounds.sigmoid_bound(p, size.e)).e
    last = np.stack([full[i, k:k + W - 1] for i, k in enumerate(n)])
    return dict(y=(np.where(on[..., None], y, 0.0), e), last=(last, np.zeros_like(last)))


def backward(x, weight, dy, bias, act, state=None, dlast=None, lengths=None):
    B, T, D = x.shape
    W, has_bias = weight.shape[1], bias is not None
    bias = np.zeros(D) if bias is None else bias
    full, on, n = _inputs(x, state, W, lengths)
    p, size = _pre(full, weight, bias, T)
    dy = np.where(on[..., None], dy, 0.0)
    q, bq = dy, Bound(dy)
    if act == "silu":
        q, bq = dy * bounds.silu_slope(p), bq * bounds.silu_slope_bound(p, size.e)
    df, m, e = np.zeros_like(full), np.zeros_like(full), np.zeros_like(full)
    for j in range(W):
        df[:, j:j + T] += weight[:, j] * q
        term = Bound(weight[:, j]) * bq
        m[:, j:j + T] += term.m
        e[:, j:j + T] += term.e
    if dlast is not None:
        for i, k in enumerate(n):
            df[i, k:k + W - 1] += dlast[i]
            m[i, k:k + W - 1] += abs(dlast[i])
    e += (W + 1) * bounds.U * m
    dweight = np.stack([(q * full[:, j:j + T]).sum((0, 1)) for j in range(W)], 1)
    ew = np.stack([(bq * Bound(full[:, j:j + T])).sum((0, 1)).e for j in range(W)], 1)
    return dict(dx=(np.where(on[..., None], df[:, W - 1:], 0.0), e[:, W - 1:]), dweight=(dweight, ew),
                dbias=(q.sum((0, 1)), bq.sum((0, 1)).e) if has_bias else None,
                dstate=None if state is None else (df[:, :W - 1], e[:, :W - 1]))
