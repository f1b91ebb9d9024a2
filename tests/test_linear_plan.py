"""Which calls of linear attention go through in segments (host code, no GPU): those that were measured faster so.  A workspace
of the forward is the segments' states."""
import ctypes

import pytest

from selective_state_space_47_amd import binding

from .test_linear_abi import lib  # noqa: F401

BF, F32 = binding.MAMBA_BF16, binding.MAMBA_F32


def cut(lib, io, batch, L, heads, dk, dv, packed=False):
    dims = binding.mamba_delta_dims(batch, L, max(heads // 4, 1), heads, dk, dv, 0, 0, 0, io, 0)
    return lib.mamba_linear_attn_workspace_bytes(ctypes.byref(dims), int(packed)) > 0


# (type, batch, tokens, heads, dk); dv = 64
WHOLE = [(F32, 8, 2048, 24, 128), (F32, 8, 2048, 32, 128), (F32, 16, 2048, 24, 128), (F32, 2, 8192, 96, 128), (F32, 8, 512, 24, 64),
         (F32, 8, 2048, 32, 64), (F32, 16, 4096, 40, 64), (BF, 8, 512, 12, 128), (BF, 8, 2048, 32, 128), (BF, 16, 2048, 24, 128),
         (BF, 8, 512, 24, 64), (BF, 16, 2048, 24, 64), (BF, 16, 4096, 40, 64)]
CUT = [(F32, 1, 2048, 12, 128), (F32, 8, 2048, 12, 128), (F32, 1, 8192, 12, 64), (F32, 8, 2048, 12, 64), (F32, 2, 8192, 96, 64),
       (BF, 1, 2048, 12, 128), (BF, 8, 2048, 12, 128), (BF, 8, 2048, 24, 128), (BF, 2, 8192, 96, 128), (BF, 1, 65536, 12, 128),
       (BF, 8, 2048, 24, 64), (BF, 2, 8192, 96, 64)]


@pytest.mark.parametrize("case", WHOLE, ids=str)
def test_whole(lib, case):
    assert not cut(lib, *case, 64)


@pytest.mark.parametrize("case", CUT, ids=str)
def test_in_segments(lib, case):
    assert cut(lib, *case, 64)


def test_packed(lib):
    for io in (BF, F32):
        assert cut(lib, io, 8, 8279, 80, 128, 64, True)
        assert not cut(lib, io, 64, 64 * 300, 600, 128, 64, True)
