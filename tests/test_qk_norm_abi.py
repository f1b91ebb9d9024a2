"""Argument checks of the norm of queries and keys that need no GPU: every invalid argument is refused before
anything is launched.  And the oracle's gradients against differences."""
import ctypes
import os

import numpy as np
import pytest

from oracle import norm
from selective_state_space_47_amd import _build, binding

FAKE = ctypes.c_void_p(0x10000)       # never dereferenced: validation fails before any launch
ODD = ctypes.c_void_p(0x10001)
HALF = ctypes.c_void_p(0x10008)
BIG = 1 << 60


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_build.LIB_PATH):
        _build.build()
    return binding.lib()


def dims(rows=4, hq=4, hk=2, d=64, rot=32, qs=0, ks=0, io=1, inter=0):
    return binding.mamba_qk_norm_rope_dims(rows, hq, hk, d, rot, qs, ks, io, inter)


def fwd(lib, dm, q=FAKE, w=FAKE, pos=FAKE, freq=FAKE, eps=1e-5, out=FAKE):
    return lib.mamba_qk_norm_rope_fwd(q, FAKE, FAKE, w, pos, freq, eps, out, FAKE,
                                      ctypes.byref(dm) if dm is not None else None, None)


def bwd(lib, dm, dout=FAKE, dk=FAKE, dw=FAKE, ws=FAKE, n=BIG):
    return lib.mamba_qk_norm_rope_bwd(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1e-5, dout, FAKE, FAKE, dk, dw, FAKE,
                                      ctypes.byref(dm) if dm is not None else None, ws, n, None)


@pytest.mark.parametrize("change,code", [
    (dict(rows=0), -2), (dict(hq=0), -2), (dict(hk=0), -2), (dict(d=0), -2), (dict(rot=-16), -2), (dict(io=2), -3),
    (dict(d=60), -4), (dict(d=264), -4), (dict(rot=24), -4), (dict(rot=80), -4), (dict(rows=1 << 31), -2),
    (dict(hq=65536), -2), (dict(hk=1 << 62), -2), (dict(qs=128), -2), (dict(ks=132), -5), (dict(qs=1 << 33), -2)],
    ids=str)
def test_dims(lib, change, code):
    dm = dims(**change)
    assert fwd(lib, dm) == code and bwd(lib, dm) == code
    assert lib.mamba_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(dm)) == 0


def test_pointers(lib):
    dm = dims()
    assert fwd(lib, None) == -1 and bwd(lib, None) == -1
    assert fwd(lib, dm, q=None) == -1 and fwd(lib, dm, w=None) == -1 and fwd(lib, dm, out=None) == -1
    assert fwd(lib, dm, pos=None) == -1 and fwd(lib, dm, freq=None) == -1
    assert fwd(lib, dm, eps=-1.0) == -4 and fwd(lib, dm, eps=float("nan")) == -4 and fwd(lib, dm, eps=float("inf")) == -4
    assert fwd(lib, dm, q=HALF) == -5 and fwd(lib, dm, w=HALF) == -5 and fwd(lib, dm, out=HALF) == -5
    assert fwd(lib, dm, pos=ctypes.c_void_p(0x10004)) == -5 and fwd(lib, dm, freq=ODD) == -5
    assert bwd(lib, dm, dout=None) == -1 and bwd(lib, dm, dk=None) == -1 and bwd(lib, dm, dw=None) == -1
    assert bwd(lib, dm, dout=HALF) == -5 and bwd(lib, dm, dw=ODD) == -5
    need = lib.mamba_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(dm))
    assert need > 0 and bwd(lib, dm, ws=None) == -6 and bwd(lib, dm, n=need - 1) == -6 and bwd(lib, dm, ws=ODD) == -5


@pytest.mark.parametrize("inter", [False, True])
def test_oracle_gradients_equal_differences(inter):
    rng = np.random.default_rng(1)
    x, w, d = rng.standard_normal((3, 2, 8)), rng.standard_normal(8), rng.standard_normal((3, 2, 8))
    pos, f = np.array([0, 5, 1000]), np.array([1.0, 0.1, 0.01])
    loss = lambda x, w: (norm.qk_norm_rope_ref(x, w, pos, f, 1e-2, inter) * d).sum()  # noqa: E731
    dx, dw = norm.qk_norm_rope_ref(x, w, pos, f, 1e-2, inter, d)
    for t, grad, f_ in ((x, dx, lambda t: loss(t, w)), (w, dw, lambda t: loss(x, t))):
        for at in np.ndindex(t.shape):
            up, down = t.copy(), t.copy()
            up[at] += 1e-5
            down[at] -= 1e-5
            assert abs((f_(up) - f_(down)) / 2e-5 - grad[at]) < 1e-8 * max(1.0, abs(grad).max())


def test_oracle_turns_by_hand():
    """Two values of mean square one, turned by a quarter."""
    x = np.array([[[np.sqrt(2.0), 0.0]]])
    out = norm.qk_norm_rope_ref(x, np.ones(2), np.array([1]), np.array([np.pi / 2]), 0.0, False)
    assert np.allclose(out, [[[0.0, np.sqrt(2.0)]]])
