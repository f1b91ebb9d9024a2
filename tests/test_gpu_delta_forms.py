"""The forms of the gated delta rule's kernels that calls with many heads take, against the fp64 oracle: passes with
workgroups of 128 columns (8 waves), chunk products that make several value heads in one workgroup, more packed
sequences than a wave has lanes, and the wide form of the segments of a long sequence.

Which form a call takes is a rule on its sizes; the rules are written out here again and each case asserts its own.
Bounds as in test_gpu_delta.py.
"""
import math
import os

import numpy as np
import pytest
import torch

from oracle import delta
from selective_state_space_47_amd import _build, binding
from tests.test_gpu_delta import BF, DEV, F32, case, check, ref_fwd, run_fwd

pytestmark = pytest.mark.gpu
GRADS = ("dq", "dk", "dv", "dg", "dbeta")


@pytest.fixture(scope="module", autouse=True)
def _native():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if not os.path.exists(_build.LIB_PATH):
        _build.build()
    binding.lib()


def wide(heads, runs, even, dv):
    """Workgroups of 128 columns: `runs` sequences or segments a head, equally long or not."""
    if dv <= 64:
        return False
    t = []
    for cols, us in ((128, 4.3), (64, 3.1)):
        rounds = heads * runs * math.ceil(dv / cols) / 256
        t.append(us * (math.ceil(rounds) if even else max(2.0, rounds)))
    return t[0] <= t[1]


def several_heads(slots, hv):
    return slots * hv > 512


# (batch, L, Hk, Hv, dk, dv): keys of the 128- and of the 64-wide tile; nine heads per key head (the gates of four are
# made at a time); columns that end inside a wave's 16
SHAPES = [(1, 70, 29, 261, 72, 128), (1, 70, 29, 174, 40, 136), (2, 129, 13, 91, 128, 120)]
ids = lambda s: "x".join(map(str, s))  # noqa: E731


def test_cases_take_these_forms():
    for B, L, Hk, Hv, dk, dv in SHAPES:
        assert wide(Hv, B, True, dv) and wide(Hv, 2 * B, True, dv)
    assert several_heads(2, 261) and several_heads(6, 91) and not several_heads(2, 174)


@pytest.mark.parametrize("io", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_many_heads(shape, io):
    x, t = case(sum(shape), *shape, io, slices=True)
    scale = shape[4] ** -0.5
    print(f"[delta forms] {shape} {io}", flush=True)
    out, last = run_fwd(t, initial_state=t["state"])
    ref, rlast = ref_fwd(x, scale, x["state"])
    check(out, ref, "out", io)
    check(last, rlast, "last_state", io, state=True)
    got = binding.mamba_delta_bwd(*(t[m] for m in ("q", "k", "v", "g", "beta", "dout")), initial_state=t["state"],
                                  dlast=t["dlast"])
    ref = delta.delta_bwd_ref(*(x[m] for m in ("q", "k", "v", "g", "beta")), scale, x["dout"], x["state"],
                              x["dlast"])
    for name in GRADS:
        check(got[name], ref[name], name, io)
    check(got["dinitial_state"], ref["dinitial_state"], "dinitial_state", io, state=True)


@pytest.mark.parametrize("io", [F32, BF], ids=["f32", "bf16"])
def test_many_packed_sequences(io):
    """More sequences than are put in order of their length, empty ones among them."""
    rng = np.random.default_rng(8)
    lengths = [int(n) for n in rng.integers(0, 40, 70)]
    lengths[3], lengths[69] = 150, 0
    total, (Hk, Hv, dk, dv) = sum(lengths), (3, 6, 64, 128)
    assert wide(Hv, 70, False, dv) and wide(Hv, 140, False, dv) and several_heads(total // 64 + 70, Hv)
    x, t = case(8, 1, total, Hk, Hv, dk, dv, io)
    for m in ("q", "k", "v", "g", "beta", "dout"):
        t[m] = t[m][0]
    st, dl = (rng.standard_normal((70, Hv, dk, dv)).astype(np.float32) for _ in range(2))
    off = np.cumsum([0] + lengths)
    kw = dict(initial_state=torch.from_numpy(st).to(DEV), seq_offsets=torch.from_numpy(off).to(DEV))
    print(f"[delta forms] {len(lengths)} sequences {io}", flush=True)
    out, last = run_fwd(t, **kw)
    got = binding.mamba_delta_bwd(*(t[m] for m in ("q", "k", "v", "g", "beta", "dout")),
                                  dlast=torch.from_numpy(dl).to(DEV), **kw)
    outs, lasts, grads = [], [], []
    for s in range(70):
        one = {m: x[m][:, off[s]:off[s + 1]] for m in ("q", "k", "v", "g", "beta", "dout")}
        o, l = ref_fwd(one, dk ** -0.5, st[s:s + 1])
        outs.append(o[0])
        lasts.append(l[0])
        grads.append(delta.delta_bwd_ref(*(one[m] for m in ("q", "k", "v", "g", "beta")), dk ** -0.5, one["dout"],
                                         st[s:s + 1], dl[s:s + 1]))
    check(out, np.concatenate(outs), "out", io)
    check(last, np.stack(lasts), "last_state", io, state=True)
    for name in GRADS:
        check(got[name], np.concatenate([r[name][0] for r in grads]), name, io)
    check(got["dinitial_state"], np.concatenate([r["dinitial_state"] for r in grads]), "dinitial_state", io,
          state=True)


@pytest.mark.parametrize("io", [F32, BF], ids=["f32", "bf16"])
def test_wide_segments(io):
    """One sequence of three heads in so many segments that their passes take 128 columns."""
    shape = B, L, Hk, Hv, dk, dv = (1, 21957, 1, 3, 64, 128)
    code = binding.MAMBA_BF16 if io == BF else binding.MAMBA_F32
    size = lambda *d: binding.mamba_delta_workspace_bytes(  # noqa: E731
        binding.mamba_delta_dims(*d, 0, 0, 0, code, 0))
    segments, rest = divmod(size(*shape) - Hv * ((L + 63) // 64) * size(1, 1, 1, 1, dk, dv),
                            Hv * dk * (dk + dv) * 4)
    assert rest == 0 and segments > 1 and wide(Hv, segments, True, dv)
    x, t = case(9, *shape, io)
    print(f"[delta forms] {segments} segments {io}", flush=True)
    out, last = run_fwd(t, initial_state=t["state"])
    ref, rlast = ref_fwd(x, dk ** -0.5, x["state"])
    check(out, ref, "out", io)
    check(last, rlast, "last_state", io, state=True)
