"""Argument checks of attention with a sliding window that need no GPU: every invalid argument is refused before
anything is launched.  And its oracle: gradients against differences, masks by hand, caches."""
import ctypes
import os

import numpy as np
import pytest

from oracle import window as ref
from selective_state_space_47_amd import _build, binding

FAKE = ctypes.c_void_p(0x10000)       # never dereferenced: validation fails before any launch
ODD = ctypes.c_void_p(0x10001)
HALF = ctypes.c_void_p(0x10008)
FOUR = ctypes.c_void_p(0x10004)
BIG = 1 << 60


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_build.LIB_PATH):
        _build.build()
    return binding.lib()


def dims(batch=2, L=100, Lk=100, Hq=4, Hk=2, d=64, qs=0, ks=0, vs=0, window=16, sinks=2, io=1):
    return binding.mamba_window_dims(batch, L, Lk, Hq, Hk, d, qs, ks, vs, window, sinks, io, 0)


def by(dm):
    return ctypes.byref(dm) if dm is not None else None


def fwd(lib, dm, q=FAKE, qo=None, ko=None, out=FAKE, lse=None):
    return lib.mamba_window_attn_fwd(q, FAKE, FAKE, qo, ko, 1.0, out, lse, by(dm), None)


def bwd(lib, dm, q=FAKE, qo=None, ko=None, out=FAKE, lse=FAKE, dout=FAKE, dq=FAKE, ws=FAKE, n=BIG):
    return lib.mamba_window_attn_bwd(q, FAKE, FAKE, qo, ko, 1.0, out, lse, dout, dq, FAKE, FAKE, by(dm), ws, n, None)


def step(lib, dm, cache=FAKE, q=FAKE, pos=FAKE, out=FAKE, ws=FAKE, n=BIG):
    return lib.mamba_window_attn_update(cache, FAKE, q, FAKE, FAKE, pos, 1.0, out, by(dm), ws, n, None)


def store(lib, dm, k=FAKE, off=None, cache=FAKE):
    return lib.mamba_window_cache_store(k, FAKE, off, cache, FAKE, by(dm), None)


BAD = [(dict(batch=0), -2), (dict(L=0), -2), (dict(Lk=0), -2), (dict(Hq=0), -2), (dict(Hk=0), -2), (dict(Hq=5), -2),
       (dict(Hq=2, Hk=4), -2), (dict(io=2), -3), (dict(d=60), -4), (dict(d=136), -4), (dict(d=0), -2), (dict(window=0), -2),
       (dict(window=1 << 41), -2), (dict(sinks=-1), -2), (dict(sinks=1 << 41), -2), (dict(L=1 << 31), -2), (dict(Lk=1 << 31), -2),
       (dict(batch=1 << 21), -2), (dict(Hq=65536, Hk=65536), -2), (dict(qs=128), -2), (dict(ks=132), -5),
       (dict(vs=1 << 23), -2), (dict(batch=1 << 20, L=1 << 30), -2), (dict(L=2 ** 63 - 1), -2)]


@pytest.mark.parametrize("change,code", BAD, ids=str)
def test_dims(lib, change, code):
    dm = dims(**change)
    assert fwd(lib, dm) == code and bwd(lib, dm) == code
    assert lib.mamba_window_attn_bwd_workspace_bytes(by(dm), 0) == 0
    one = dims(**{"L": 1, "Lk": 1, **change})
    assert step(lib, one) == code
    assert lib.mamba_window_attn_update_workspace_bytes(by(one)) == 0
    if not set(change) & {"L", "Hq", "qs"}:  # (a store does not look at the queries' sizes)
        assert store(lib, dm) == code


def test_pointers(lib):
    assert fwd(lib, None) == -1 and bwd(lib, None) == -1 and step(lib, None) == -1 and store(lib, None) == -1
    dm, one = dims(), dims(L=1, Lk=1, window=1000)
    for call, m in ((fwd, dm), (bwd, dm), (step, one)):
        assert call(lib, m, q=None) == -1 and call(lib, m, q=HALF) == -5
        assert call(lib, m, out=None) == -1 and call(lib, m, out=ODD) == -5
    for call in (fwd, bwd):
        assert call(lib, dm, qo=FAKE) == -1 and call(lib, dm, ko=FAKE) == -1 and call(lib, dm, qo=FOUR, ko=FAKE) == -5
    assert fwd(lib, dm, lse=ODD) == -5
    assert bwd(lib, dm, lse=None) == -1 and bwd(lib, dm, dout=None) == -1 and bwd(lib, dm, dq=None) == -1
    assert bwd(lib, dm, dout=HALF) == -5 and bwd(lib, dm, ws=None) == -6 and bwd(lib, dm, ws=HALF) == -5
    assert bwd(lib, dm, n=lib.mamba_window_attn_bwd_workspace_bytes(by(dm), 0) - 1) == -6
    assert step(lib, one, cache=None) == -1 and step(lib, one, pos=None) == -1 and step(lib, one, cache=HALF) == -5
    assert step(lib, one, pos=FOUR) == -5 and step(lib, dims(L=2, Lk=1)) == -2 and step(lib, dims(L=1, Lk=2)) == -2
    need = lib.mamba_window_attn_update_workspace_bytes(by(one))
    assert need > 0 and step(lib, one, ws=None) == -6 and step(lib, one, n=need - 1) == -6 and step(lib, one, ws=HALF) == -5
    assert store(lib, dm, k=None) == -1 and store(lib, dm, cache=None) == -1 and store(lib, dm, k=HALF) == -5
    assert store(lib, dm, cache=HALF) == -5 and store(lib, dm, off=FOUR) == -5
    # caches past the addresses' bound
    assert store(lib, dims(window=1 << 40)) == -2 and step(lib, dims(L=1, Lk=1, window=1 << 40)) == -2


def test_oracle_masks_by_hand():
    see = ref.visible(4, 6, 2, 1)  # positions 2 .. 5, two last keys and the first
    assert see.tolist() == [[True, True, True, False, False, False], [True, False, True, True, False, False],
                            [True, False, False, True, True, False], [True, False, False, False, True, True]]
    assert ref.visible(3, 1, 5, 0).tolist() == [[False], [False], [True]]


def test_oracle_gradients_equal_differences():
    rng = np.random.default_rng(0)
    x = dict(q=rng.standard_normal((7, 4, 3)), k=rng.standard_normal((6, 2, 3)), v=rng.standard_normal((6, 2, 3)))
    do = rng.standard_normal((7, 4, 3))
    loss = lambda x: (ref.window_ref(x["q"], x["k"], x["v"], 3, 1, 0.7)[0] * do).sum()  # noqa: E731
    grads = ref.window_ref(x["q"], x["k"], x["v"], 3, 1, 0.7, do)
    for m, g in zip("qkv", grads):
        for at in np.ndindex(x[m].shape):
            up, down = x[m].copy(), x[m].copy()
            up[at] += 1e-5
            down[at] -= 1e-5
            assert abs((loss({**x, m: up}) - loss({**x, m: down})) / 2e-5 - g[at]) < 1e-8


def test_oracle_caches_hold_what_a_query_sees():
    for window, sinks in ((3, 2), (4, 0), (1, 1)):
        for n in range(1, 15):
            pos = np.arange(n, dtype=float)[:, None, None] + 1.0
            kept = set(ref.store_ref(np.zeros((window + sinks, 1, 1)), pos, window, sinks)[:, 0, 0]) - {0.0}
            assert kept == set(pos[ref.visible(n, n, window, sinks)[-1], 0, 0])
