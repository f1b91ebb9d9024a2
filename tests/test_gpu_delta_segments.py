"""Long sequences of few heads, which go through in segments side by side: the last state written over the initial
one.  (Which workgroup runs first is not fixed, so that a workgroup that still read the initial state from there
would fail this now and then only; that none does is in the kernels: the output pass starts every segment, the first
too, from the workspace.)"""
import os

import numpy as np
import pytest
import torch

from selective_state_space_47_amd import _build, binding
from tests.test_gpu_delta import BF, DEV, F32, case, check, ref_fwd, run_fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _native():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if not os.path.exists(_build.LIB_PATH):
        _build.build()
    binding.lib()


def segmented(io, B, L, Hv, dk, dv, packed):
    """Whether such a call holds more than the chunk products in its workspace."""
    code = binding.MAMBA_BF16 if io == BF else binding.MAMBA_F32
    dm = binding.mamba_delta_dims(B, L, 1, Hv, dk, dv, 0, 0, 0, code, 0)
    one = binding.mamba_delta_dims(1, 1, 1, 1, dk, dv, 0, 0, 0, code, 0)
    slots = L // 64 + B if packed else B * ((L + 63) // 64)
    return binding.mamba_delta_workspace_bytes(dm, packed) > slots * Hv * binding.mamba_delta_workspace_bytes(one)


# a last segment of one token, of a whole chunk, of several; columns that do not fill a block
@pytest.mark.parametrize("io", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 4097, 1, 2, 64, 64), (2, 4160, 1, 1, 128, 136), (1, 5000, 1, 2, 40, 24)],
                         ids=lambda s: "x".join(map(str, s)))
def test_state_in_place(shape, io):
    B, L, _, Hv, dk, dv = shape
    assert segmented(io, B, L, Hv, dk, dv, False)
    x, t = case(L, *shape, io)
    print(f"[delta segments] {shape} {io}", flush=True)
    out, last = run_fwd(t, initial_state=t["state"])
    check(last, ref_fwd(x, dk ** -0.5, x["state"])[1], "last_state", io, state=True)
    for _ in range(5):
        st = t["state"].clone()
        got, same = run_fwd(t, initial_state=st, last_state=st)
        assert same is st and torch.equal(got, out) and torch.equal(st, last)


@pytest.mark.parametrize("io", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("state", [True, False], ids=["state", "zero"])
def test_packed_states_in_place(io, state):
    """Sequences of no, one and several segments; and from zero with a state that is only written."""
    lengths = [4097, 0, 1, 2500, 64, 0]
    Hv, dk, dv = 2, 64, 72
    assert segmented(io, len(lengths), sum(lengths), Hv, dk, dv, True)
    x, t = case(7, 1, sum(lengths), 1, Hv, dk, dv, io)
    args = {m: t[m][0] for m in ("q", "k", "v", "g", "beta")}
    st = np.random.default_rng(9).standard_normal((len(lengths), Hv, dk, dv)).astype(np.float32)
    st = st if state else np.zeros_like(st)
    off = np.cumsum([0] + lengths)
    toff = torch.from_numpy(off).to(DEV)
    print(f"[delta segments] packed {io} {state}", flush=True)
    ref = [ref_fwd({m: x[m][:, off[s]:off[s + 1]] for m in args}, dk ** -0.5, st[s:s + 1])
           for s in range(len(lengths))]
    for _ in range(3):
        buf = torch.from_numpy(st).to(DEV)
        out, last = run_fwd(args, initial_state=buf if state else None, last_state=buf, seq_offsets=toff)
        assert last is buf
        check(out, np.concatenate([r[0][0] for r in ref]), "out", io)
        check(buf, np.concatenate([r[1] for r in ref]), "last_state", io, state=True)
        for s in (1, 5):
            assert np.array_equal(buf[s].cpu().numpy(), st[s])
