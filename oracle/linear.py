"""fp64 reference of linear attention with a decay per head and its gradients (test infrastructure only).

Written token by token from the recurrence, per value head with the key head it shares:
    S_t = exp(g_t) S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t
and, for the gradients, from its adjoint.  Pinned by the oracle linear tests: the gradients equal central finite
differences of the forward, and the outputs the sum over pairs of tokens.
"""
from __future__ import annotations

import numpy as np

from .delta import _decay, _heads


def linear_ref(q, k, v, g, scale, state=None, keep=None):
    """One batch of equally long sequences: q, k (B, L, Hk, dk), v (B, L, Hv, dv), g (B, L, Hv).  Returns
    (out, last state).  `keep`: a list that receives the state after every token."""
    B, L, Hv, dv = v.shape
    dk, rep = k.shape[-1], Hv // k.shape[-2]
    q, k, v, a = _heads(q, rep), _heads(k, rep), np.asarray(v, dtype=np.float64), _decay(g)
    S = np.zeros((B, Hv, dk, dv)) if state is None else np.array(state, dtype=np.float64)
    out = np.zeros((B, L, Hv, dv))
    for t in range(L):
        S = a[:, t, :, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        out[:, t] = scale * np.einsum("bhkv,bhk->bhv", S, q[:, t])
        if keep is not None:
            keep.append(S)
    return out, S


def linear_bwd_ref(q, k, v, g, scale, dout, state=None, dlast=None):
    """Gradients for the loss sum(out * dout) + sum(last * dlast): a dict like the library's."""
    B, L, Hv, dv = v.shape
    Hk, dk = k.shape[-2:]
    rep = Hv // Hk
    states = []
    linear_ref(q, k, v, g, scale, state, states)
    S0 = np.zeros((B, Hv, dk, dv)) if state is None else np.array(state, dtype=np.float64)
    q, k, v, a = _heads(q, rep), _heads(k, rep), np.asarray(v, dtype=np.float64), _decay(g)
    dout = np.asarray(dout, dtype=np.float64)
    lam = np.zeros((B, Hv, dk, dv)) if dlast is None else np.array(dlast, dtype=np.float64)
    dq, dkk, dvv, dg = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros((B, L, Hv))
    for t in reversed(range(L)):
        do = scale * dout[:, t]
        dq[:, t] = np.einsum("bhkv,bhv->bhk", states[t], do)
        lam = lam + q[:, t, :, :, None] * do[:, :, None, :]
        dkk[:, t] = np.einsum("bhkv,bhv->bhk", lam, v[:, t])
        dvv[:, t] = np.einsum("bhkv,bhk->bhv", lam, k[:, t])
        lam = a[:, t, :, None, None] * lam
        dg[:, t] = (lam * (states[t - 1] if t else S0)).sum((-1, -2))
    group = lambda x: x.reshape(B, L, Hk, rep, dk).sum(3)  # noqa: E731
    return dict(dq=group(dq), dk=group(dkk), dv=dvv, dg=dg, dinitial_state=lam)
