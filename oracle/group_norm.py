"""Group norm with an activation or a gate, channels last, in fp64 (test oracle)."""
from __future__ import annotations

import math

import numpy as np

# Phi(z) by erfc, which keeps its digits far below zero, where 1 + erf would cancel
_phi = np.vectorize(lambda z: 0.5 * math.erfc(-z / math.sqrt(2)), otypes=[np.float64])


def act(z, kind):
    if kind == "silu":
        return z / (1 + np.exp(-z))
    if kind == "gelu":
        return z * _phi(z)
    return z


def slope(z, kind):
    if kind == "silu":
        s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    if kind == "gelu":
        return _phi(z) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return np.ones_like(z)


def _parts(x, groups, w, b, lengths, eps):
    """Per n: (rows that count, xhat [L, C], z, m [G], r [G])."""
    N, S, C = x.shape
    for n in range(N):
        L = S if lengths is None else int(min(max(int(lengths[n]), 0), S))
        xg = np.asarray(x[n, :L], np.float64).reshape(L, groups, C // groups)
        m = xg.mean((0, 2)) if L else np.zeros(groups)
        var = ((xg - m[:, None]) ** 2).mean((0, 2)) if L else np.zeros(groups)
        r = 1 / np.sqrt(var + eps)
        hat = ((xg - m[:, None]) * r[:, None]).reshape(L, C)
        yield n, L, hat, hat * w + b, m, r


def forward(x, groups, weight=None, bias=None, gate=None, kind="silu", eps=1e-5, lengths=None):
    """x [N, S, C] -> (y, stats [N, groups, 2])."""
    N, S, C = x.shape
    w = np.ones(C) if weight is None else weight
    b = np.zeros(C) if bias is None else bias
    y, stats = np.zeros((N, S, C)), np.zeros((N, groups, 2))
    for n, L, _, z, m, r in _parts(x, groups, w, b, lengths, eps):
        stats[n, :, 0], stats[n, :, 1] = m, r
        y[n, :L] = act(z, kind) if gate is None else z * act(np.asarray(gate[n, :L], np.float64), kind)
    return y, stats


def backward(x, dy, groups, weight=None, bias=None, gate=None, kind="silu", eps=1e-5, lengths=None):
    """(dx, dweight, dbias, dgate) of sum(y * dy)."""
    N, S, C = x.shape
    w = np.ones(C) if weight is None else weight
    b = np.zeros(C) if bias is None else bias
    dx, dw, db = np.zeros((N, S, C)), np.zeros(C), np.zeros(C)
    dgate = None if gate is None else np.zeros((N, S, C))
    for n, L, hat, z, _, r in _parts(x, groups, w, b, lengths, eps):
        if not L:
            continue
        d = np.asarray(dy[n, :L], np.float64)
        if gate is None:
            dz = d * slope(z, kind)
        else:
            q = np.asarray(gate[n, :L], np.float64)
            dz = d * act(q, kind)
            dgate[n, :L] = d * z * slope(q, kind)
        dw += (dz * hat).sum(0)
        db += dz.sum(0)
        g, h = (dz * w).reshape(L, groups, C // groups), hat.reshape(L, groups, C // groups)
        dx[n, :L] = ((g - g.mean((0, 2), keepdims=True) - h * (g * h).mean((0, 2), keepdims=True))
                     * r[:, None]).reshape(L, C)
    return dx, dw, db, dgate
