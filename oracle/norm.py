"""fp64 reference of the norms around a block and of their gradients (test infrastructure only)."""
from __future__ import annotations

import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def _rms(a, eps):
    return 1.0 / np.sqrt((a * a).mean(-1, keepdims=True) + eps)


def _silu(z):
    s = 1.0 / (1.0 + np.exp(-z))
    return z * s, s * (1.0 + z * (1.0 - s))


def _norm_bwd(a, w, d, eps):
    """Gradient of a * rms(a) * w for the output gradient d, and the normed a."""
    r = _rms(a, eps)
    h = a * r
    return r * (d * w - h * (d * w * h).mean(-1, keepdims=True)), h


def gated_norm_ref(y, z, weight, eps, gate_first, dout=None):
    """out, or the dict of gradients for dout.  y, z: (rows, groups, dim); weight (dim,) or
    (groups, dim)."""
    y, z, w, d = _f64(y), _f64(z), _f64(weight), _f64(dout)
    gate, slope = (np.ones_like(y), np.zeros_like(y)) if z is None else _silu(z)
    a = y * gate if gate_first else y
    if dout is None:
        n = a * _rms(a, eps) * w
        return n if gate_first else n * gate
    over = (0,) if w.ndim == 2 else (0, 1)
    if gate_first:
        da, h = _norm_bwd(a, w, d, eps)
        return dict(dy=da * gate, dz=None if z is None else da * y * slope,
                    dweight=(d * h).sum(over))
    da, h = _norm_bwd(y, w, d * gate, eps)
    return dict(dy=da, dz=None if z is None else d * h * w * slope,
                dweight=(d * gate * h).sum(over))


def add_norm_ref(x, residual, weight, scale, post, eps, dout=None, dres=None):
    """(out, r), or the dict of gradients for dout and dres."""
    x, q, w, s, p = (_f64(t) for t in (x, residual, weight, scale, post))
    n = x if p is None else x * _rms(x, eps) * p
    r = (0.0 if q is None else q) + (n if s is None else s * n)
    if dout is None:
        return r * _rms(r, eps) * w, r
    d = _f64(dout)
    dr, h = _norm_bwd(r, w, d, eps)
    if dres is not None:
        dr = dr + _f64(dres)
    dn = dr if s is None else dr * s
    g = dict(dresidual=None if q is None else dr, dweight=(d * h).sum(0),
             dscale=None if s is None else (dr * n).sum(0), dx=dn, dpost_weight=None)
    if p is not None:
        g["dx"], h = _norm_bwd(x, p, dn, eps)
        g["dpost_weight"] = (dn * h).sum(0)
    return g


def qk_norm_rope_ref(x, weight, positions, inv_freq, eps, interleaved, dout=None):
    """The norm per head and the rotation of x (rows, heads, dim): out, or (dx, dweight) for dout."""
    x, w, f = _f64(x), _f64(weight), _f64(inv_freq)
    half = len(f)
    angle = np.asarray(positions, dtype=np.float64)[:, None, None] * f
    c, s = np.cos(angle), np.sin(angle)
    i = np.arange(half)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)

    def turn(h, s):
        out = h.copy()
        out[..., one] = h[..., one] * c - h[..., two] * s
        out[..., two] = h[..., two] * c + h[..., one] * s
        return out

    if dout is None:
        return turn(x * _rms(x, eps) * w, s)
    dh = turn(_f64(dout), -s)
    dx, n = _norm_bwd(x, w, dh, eps)
    return dx, (dh * n).sum((0, 1))
