"""How exact linear attention is with bf16 storage, each result being the fp32 one rounded once, and how far a NaN or an
infinity reaches inside a sequence.

With x the kernel's value before its rounding, w the exact one and r(x) the distance of x to the bf16 it becomes: r changes
by at most |x - w| between x and w, so that |bf16(x) - w| <= r(w) + 2 |x - w|, value by value and in the 2-norm.  r(w) is
computed here from the exact value.  |x - w| is 2e-5 of the norm, as with fp32 storage, and 2^-17 of it from each factor that
is two bf16 parts (two of them at most are in one product).  Value by value it is that of the sizes of the value's terms, which
are the same sums of the factors' absolute values.
"""
import numpy as np
import pytest
import torch

from oracle import linear

from .test_gpu_linear import BF, CUT, DEV, F32, IO, _native, case, ids, packed_case, ref_fwd, run_fwd  # noqa: F401
from .test_gpu_linear_bwd import ref_bwd, run_bwd

pytestmark = pytest.mark.gpu
FP32, PARTS = 2e-5, 2.0 ** -16
BF_GRADS = ("dq", "dk", "dv")


def rounded_once(got, want, sizes, name):
    got, want = got.double().cpu().numpy(), np.asarray(want)
    assert np.isfinite(got).all(), name
    own = torch.from_numpy(want).to(BF).double().numpy() - want
    size, off = np.linalg.norm(want), np.linalg.norm(got - want)
    print(f"[linear once] {name}: {off / size:.3e}, rounding {np.linalg.norm(own) / size:.3e}", flush=True)
    assert off <= np.linalg.norm(own) + 2 * (FP32 + PARTS) * size, name
    assert (np.abs(got - want) <= np.abs(own) + 2 * (FP32 + PARTS) * sizes).all(), name


def sizes_of(x):
    return {m: np.abs(a) if m != "g" else a for m, a in x.items()}


# (batch, L, Hk, Hv, dk, dv): several chunks and units, heads that do not fill a tile, several column blocks, segments
SHAPES = [(2, 64, 1, 2, 128, 64), (3, 130, 1, 3, 40, 72), (1, 257, 2, 2, 128, 64), (1, 333, 1, 2, 72, 264),
          (1, 2600, 1, 1, 64, 64)]


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_out_and_gradients_round_once(shape):
    x, t = case(sum(shape) + 3, *shape, BF)
    scale, size = shape[4] ** -0.5, sizes_of(x)
    out, _ = run_fwd(t, initial_state=t["state"])
    rounded_once(out, ref_fwd(x, scale, x["state"])[0], ref_fwd(size, scale, size["state"])[0], "out")
    got = run_bwd(t, initial_state=t["state"], dlast=t["dlast"])
    want = ref_bwd(x, scale, x["state"], x["dlast"])
    most = ref_bwd(size, scale, size["state"], size["dlast"])
    for name in BF_GRADS:
        rounded_once(got[name], want[name], most[name], name)


def test_packed_partly_cut_rounds_once():
    x, t, off, one, _ = packed_case(CUT, BF, Hk=2, Hv=40, dk=24, dv=16)
    out, _ = run_fwd(t, initial_state=t["state"], seq_offsets=off)
    got = run_bwd(t, initial_state=t["state"], dlast=t["dlast"], seq_offsets=off)
    scale, size = 24 ** -0.5, sizes_of(x)
    refs, most = [], []
    for s in range(len(CUT)):
        mine, theirs = one(s), sizes_of(one(s))
        refs.append(dict(ref_bwd(mine, scale, x["state"][s:s + 1], x["dlast"][s:s + 1]),
                         out=ref_fwd(mine, scale, x["state"][s:s + 1])[0]))
        most.append(dict(ref_bwd(theirs, scale, size["state"][s:s + 1], size["dlast"][s:s + 1]),
                         out=ref_fwd(theirs, scale, size["state"][s:s + 1])[0]))
    for name in ("out", *BF_GRADS):
        a = out if name == "out" else got[name]
        rounded_once(a[3:], *(np.concatenate([r[name][0] for r in rs]) for rs in (refs, most)), name)


def same(a, b, keep):
    return torch.equal(a[keep], b[keep])


@IO
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
@pytest.mark.parametrize("lengths", [[70, 500, 90], [10, 9000]], ids=lambda v: "-".join(map(str, v)))
def test_reach_of_nan_and_infinity_forward(lengths, bad, io):
    """In q: the outputs of its chunk of 64 tokens at most; in k and v: of its chunk and what follows; never an earlier
    chunk, another sequence, or (in v) another value head or column.  (9000 tokens of two heads go through in segments.)"""
    x, t, off, _, total = packed_case(lengths, io, Hk=1, Hv=2, dk=64, dv=64)
    first = int(off[1])          # of the second sequence
    at, chunk = first + 200, first + 192
    print(f"[linear reach] {lengths} {bad} {io}", flush=True)
    clean, last = run_fwd(t, seq_offsets=off)
    token = torch.arange(total, device=DEV)
    held = token >= int(off[0])  # (the gap before the first sequence is not written)
    other = ((token < first) | (token >= int(off[2]))) & held
    for m in ("q", "k", "v"):
        row = t[m].clone()
        row[at, 0, 5] = bad
        out, state = run_fwd({**t, m: row}, seq_offsets=off)
        assert same(out, clean, other) and torch.equal(state[0], last[0]), m
        assert same(out, clean, held & (token < chunk)), m
        assert not bool(torch.isfinite(out[at, 0]).all()), m
        if m == "q":
            assert same(out, clean, held & (token >= chunk + 64)) and torch.equal(state, last)
        if m == "v":
            cols = torch.arange(64, device=DEV) != 5
            assert same(out[:, 0][:, cols], clean[:, 0][:, cols], held) and same(out[:, 1], clean[:, 1], held)


@IO
@pytest.mark.parametrize("lengths", [[70, 700, 90], [10, 9000]], ids=lambda v: "-".join(map(str, v)))
def test_reach_of_nan_in_the_gradients(lengths, io):
    """A NaN in v reaches dk and dg of its block of 128 tokens (fp32 storage: 64) and, through the state, dq and dg of
    what follows; one in dout dq of its block and, through the adjoint, dk, dv and dg of what is before it; no other
    sequence's."""
    x, t, off, _, total = packed_case(lengths, io, Hk=1, Hv=2, dk=64, dv=64)
    unit, first = 128 if io == BF else 64, int(off[1])
    at = first + 300
    lo = first + 300 // unit * unit
    hi = lo + unit
    print(f"[linear reach bwd] {lengths} {io}", flush=True)
    clean = run_bwd(t, seq_offsets=off)
    token = torch.arange(total, device=DEV)
    held = token >= int(off[0])
    other = ((token < first) | (token >= int(off[2]))) & held
    before, behind = held & (token < lo), held & (token >= hi)
    for m, kept in (("v", dict(dq=before, dk=before | behind, dv=held, dg=before)),
                    ("dout", dict(dq=before | behind, dk=behind, dv=behind, dg=behind))):
        row = t[m].clone()
        row[at, 0, 5] = float("nan")
        got = run_bwd({**t, m: row}, seq_offsets=off)
        for name, keep in kept.items():
            assert same(got[name], clean[name], other) and same(got[name], clean[name], keep), (m, name)
