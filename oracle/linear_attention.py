"""Linear attention with a decay for each head, token by token in fp64 (test oracle).

S_t = g S_(t-1) + k_t v_t^T, o_t = scale S_t^T q_t with g = exp(log_decay), head by head; the backward pass by the
reversed recurrence R_t = g R_(t+1) + scale q_t do_t^T.  Tokens at and behind lengths[b] do not exist.
"""
from __future__ import annotations

import numpy as np


def _decay(log_decay):
    return np.exp(np.asarray(log_decay, np.float64))[:, None, None]


def _length(lengths, b, T):
    return T if lengths is None else int(min(max(int(lengths[b]), 0), T))


def forward(q, k, v, log_decay, s0=None, lengths=None, scale=1.0):
    """q [B,T,H,dk], k [B,T,Hkv,dk], v [B,T,Hkv,dv] -> (o [B,T,H,dv], s [B,H,dk,dv])."""
    B, T, H, dk = q.shape
    dv, per, g = v.shape[3], H // k.shape[2], _decay(log_decay)
    o = np.zeros((B, T, H, dv))
    s = np.zeros((B, H, dk, dv)) if s0 is None else np.array(s0, np.float64)
    for b in range(B):
        for t in range(_length(lengths, b, T)):
            kt, vt = np.repeat(k[b, t], per, 0), np.repeat(v[b, t], per, 0)
            s[b] = g * s[b] + kt[:, :, None] * vt[:, None, :]
            o[b, t] = scale * np.einsum("hi,hij->hj", q[b, t], s[b])
    return o, s


def backward(q, k, v, log_decay, do, s0=None, ds=None, lengths=None, scale=1.0):
    """(dq, dk, dv, ds0) of sum(o * do) + sum(s * ds)."""
    B, T, H, dk = q.shape
    Hkv, dv = k.shape[2], v.shape[3]
    per, g = H // Hkv, _decay(log_decay)
    dq, dkk, dvv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    ds0 = np.zeros((B, H, dk, dv))
    for b in range(B):
        L = _length(lengths, b, T)
        s = np.zeros((H, dk, dv)) if s0 is None else np.array(s0[b], np.float64)
        for t in range(L):
            kt, vt = np.repeat(k[b, t], per, 0), np.repeat(v[b, t], per, 0)
            s = g * s + kt[:, :, None] * vt[:, None, :]
            dq[b, t] = scale * np.einsum("hij,hj->hi", s, do[b, t])
        r = np.zeros((H, dk, dv)) if ds is None else np.array(ds[b], np.float64)
        for t in range(L - 1, -1, -1):
            kt, vt = np.repeat(k[b, t], per, 0), np.repeat(v[b, t], per, 0)
            r = r + scale * q[b, t][:, :, None] * do[b, t][:, None, :]
            dkk[b, t] = np.einsum("hij,hj->hi", r, vt).reshape(Hkv, per, dk).sum(1)
            dvv[b, t] = np.einsum("hij,hi->hj", r, kt).reshape(Hkv, per, dv).sum(1)
            r = g * r
        ds0[b] = r
    return dq, dkk, dvv, ds0


def step(q, k, v, log_decay, state, slots=None, scale=1.0):
    """One token: (o [B,H,dv], the states after it); rows of one slot in row order."""
    B, H, dk = q.shape
    per, g = H // k.shape[1], _decay(log_decay)
    after, o = np.array(state, np.float64), np.zeros((B, H, v.shape[2]))
    for b in range(B):
        i = b if slots is None else int(slots[b])
        if 0 <= i < len(after):
            kt, vt = np.repeat(k[b], per, 0), np.repeat(v[b], per, 0)
            after[i] = g * after[i] + kt[:, :, None] * vt[:, None, :]
            o[b] = scale * np.einsum("hi,hij->hj", q[b], after[i])
    return o, after
