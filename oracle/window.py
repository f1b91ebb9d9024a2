"""fp64 reference of causal attention with a sliding window and sinks, its gradients and its ring caches (test
infrastructure only).

The query at position p sees key j where j <= p and (p - j < window or j < sinks):
    out = softmax(scale q . k) v over the keys that it sees, zero where it sees none
Pinned by the oracle window tests: the gradients equal central finite differences, hand-worked masks, and the caches
hold what a query sees.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def visible(n, m, window, sinks):
    """(n, m): which of m keys each of the last n tokens sees."""
    p, j = np.arange(n)[:, None] + (m - n), np.arange(m)[None, :]
    return (j <= p) & ((p - j < window) | (j < sinks))


def window_ref(q, k, v, window, sinks, scale, dout=None):
    """One sequence, q (n, Hq, d), k, v (m, Hk, d): (out, lse), or with dout (dq, dk, dv)."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    (n, Hq, d), (m, Hk) = q.shape, k.shape[:2]
    rep, see = Hq // Hk, visible(n, m, window, sinks)
    out, lse = np.zeros_like(q), np.full((n, Hq), -np.inf)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    some = see.any(1)
    for h in range(Hq):
        K, V = k[:, h // rep], v[:, h // rep]
        s = np.where(see, scale * (q[:, h] @ K.T), -np.inf)
        top = np.where(some, s.max(1, initial=-np.inf), 0.0)
        e = np.exp(s - top[:, None])
        sums = e.sum(1)
        P = e / np.where(some, sums, 1.0)[:, None]
        out[:, h] = P @ V
        lse[some, h] = top[some] + np.log(sums[some])
        if dout is not None:
            do = _f64(dout)[:, h]
            dp = do @ V.T
            ds = scale * P * (dp - (P * dp).sum(1, keepdims=True))
            dv[:, h // rep] += P.T @ do
            dq[:, h] = ds @ K
            dk[:, h // rep] += ds.T @ q[:, h]
    return (out, lse) if dout is None else (dq, dk, dv)


def slot(p, window, sinks):
    return p if p < sinks else sinks + (p - sinks) % window


def store_ref(cache, x, window, sinks):
    """cache (slots, Hk, d) with the tokens x (m, Hk, d) of a sequence put in one after another."""
    cache = np.array(cache)
    for p in range(len(x)):
        cache[slot(p, window, sinks)] = x[p]
    return cache
