"""fp64 reference of the gated delta rule and its gradients (test infrastructure only).

Written token by token from the recurrence, per value head with the key head it shares:
    S~ = exp(g_t) S,  e = v_t - S~^T k_t,  S = S~ + beta_t k_t e^T,  o_t = scale S^T q_t
and, for the gradients, from its adjoint.  Pinned by the oracle delta tests: the gradients equal central
finite differences of the forward, and hand-worked cases.
"""
from __future__ import annotations

import numpy as np


def _heads(x, rep):
    return np.repeat(np.asarray(x, dtype=np.float64), rep, axis=-2)


def _decay(g):
    with np.errstate(over="ignore"):
        return np.exp(np.asarray(g, dtype=np.float64))


def delta_ref(q, k, v, g, beta, scale, state=None, keep=None):
    """One batch of equally long sequences: q, k (B, L, Hk, dk), v (B, L, Hv, dv), g, beta (B, L, Hv).
    Returns (out, last state).  `keep`: a list that receives the state after every token."""
    B, L, Hv, dv = v.shape
    dk, rep = k.shape[-1], Hv // k.shape[-2]
    q, k, v = _heads(q, rep), _heads(k, rep), np.asarray(v, dtype=np.float64)
    a, beta = _decay(g), np.asarray(beta, dtype=np.float64)
    S = np.zeros((B, Hv, dk, dv)) if state is None else np.array(state, dtype=np.float64)
    out = np.zeros((B, L, Hv, dv))
    for t in range(L):
        S = a[:, t, :, None, None] * S
        e = v[:, t] - np.einsum("bhkv,bhk->bhv", S, k[:, t])
        S = S + (beta[:, t, :, None] * k[:, t])[..., None] * e[:, :, None, :]
        out[:, t] = scale * np.einsum("bhkv,bhk->bhv", S, q[:, t])
        if keep is not None:
            keep.append(S)
    return out, S


def delta_bwd_ref(q, k, v, g, beta, scale, dout, state=None, dlast=None):
    """Gradients for the loss sum(out * dout) + sum(last * dlast): a dict like the library's."""
    B, L, Hv, dv = v.shape
    Hk, dk = k.shape[-2:]
    rep = Hv // Hk
    states = []
    delta_ref(q, k, v, g, beta, scale, state, states)
    S0 = np.zeros((B, Hv, dk, dv)) if state is None else np.array(state, dtype=np.float64)
    q, k, v = _heads(q, rep), _heads(k, rep), np.asarray(v, dtype=np.float64)
    a, beta, dout = _decay(g), np.asarray(beta, dtype=np.float64), np.asarray(dout, dtype=np.float64)
    lam = np.zeros((B, Hv, dk, dv)) if dlast is None else np.array(dlast, dtype=np.float64)
    dq, dkk = np.zeros((B, L, Hv, dk)), np.zeros((B, L, Hv, dk))
    dvv, dg, db = np.zeros((B, L, Hv, dv)), np.zeros((B, L, Hv)), np.zeros((B, L, Hv))
    for t in reversed(range(L)):
        before = states[t - 1] if t else S0
        X = a[:, t, :, None, None] * before
        e = v[:, t] - np.einsum("bhkv,bhk->bhv", X, k[:, t])
        do = scale * dout[:, t]
        dq[:, t] = np.einsum("bhkv,bhv->bhk", states[t], do)
        lam = lam + q[:, t, :, :, None] * do[:, :, None, :]
        lk = np.einsum("bhkv,bhk->bhv", lam, k[:, t])      # adjoint of beta e
        b = beta[:, t, :, None]
        de = b * lk
        dkk[:, t] = np.einsum("bhkv,bhv->bhk", lam, b * e) - np.einsum("bhkv,bhv->bhk", X, de)
        dvv[:, t] = de
        db[:, t] = (lk * e).sum(-1)
        lam = lam - k[:, t, :, :, None] * de[:, :, None, :]
        dg[:, t] = (lam * X).sum((-1, -2))
        lam = a[:, t, :, None, None] * lam
    group = lambda x: x.reshape(B, L, Hk, rep, dk).sum(3)  # noqa: E731
    return dict(dq=group(dq), dk=group(dkk), dv=dvv, dg=dg, dbeta=db, dinitial_state=lam)
