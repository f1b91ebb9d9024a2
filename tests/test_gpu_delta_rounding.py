"""bf16 calls of the gated delta rule round each result once: their error against fp64 is that of rounding the
fp64 result to bf16.

Bound: with |.| the 2-norm over a tensor and round() the rounding to bf16, |x - ref| <= 1.1 |round(ref) - ref|.
Before its rounding a result differs from ref by d: each product's factors are held to 2^-17 (two bf16 parts),
four of them in a row at most, 3e-5 of the products' size.  Rounding ref + d instead of ref moves a value by
at most 2 d more than ref's own rounding, and |round(ref) - ref| is 1.66e-3 |ref|, so that 2 d is below 0.04 of it
where the products do not cancel, and the bound leaves room for results that are less than half their products'
size.  A factor in one bf16 part adds as much again as the result's own rounding: 1.4 of it.
"""
import os

import numpy as np
import pytest
import torch

from oracle import delta
from selective_state_space_47_amd import _build, binding, synth
from tests.test_gpu_delta import BF, DEV, case, ref_fwd, run_fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _native():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if not os.path.exists(_build.LIB_PATH):
        _build.build()
    binding.lib()


def check(got, ref, name, bound=1.1):
    ref = np.asarray(ref, np.float64)
    once = np.linalg.norm(synth.round_to_bf16(ref.astype(np.float32)).astype(np.float64) - ref)
    off = np.linalg.norm(got.double().cpu().numpy() - ref)
    print(f"[delta rounding] {name}: {off / once:.3f} of one rounding", flush=True)
    assert off <= bound * once, name


# key heads, value heads, dk, dv: the smallest tile of keys and the largest, columns of one block and of several
HEADS = [(2, 4, 128, 128), (3, 6, 64, 64), (1, 2, 72, 264)]


def inputs(heads, aligned):
    """`aligned`: queries near the keys and decays near one, as in a model that reads back what it stored: what the
    state holds for a token's key is then most of its output, instead of a sum of independent terms."""
    x, t = case(sum(heads), 2, 200, *heads, BF)
    if aligned:
        near = x["k"] + 0.02 * np.random.default_rng(1).standard_normal(x["k"].shape).astype(np.float32)
        for m, v in (("q", near), ("g", 0.02 * x["g"])):
            x[m] = synth.round_to_bf16(v)
            t[m] = torch.from_numpy(x[m]).to(DEV).to(BF)
    return x, t


@pytest.mark.parametrize("aligned", [False, True], ids=["random", "aligned"])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "x".join(map(str, h)))
def test_output(heads, aligned):
    x, t = inputs(heads, aligned)
    print(f"[delta rounding] {heads} aligned={aligned}", flush=True)
    for state in (None, "state"):
        out, _ = run_fwd(t, initial_state=state and t[state])
        check(out, ref_fwd(x, heads[2] ** -0.5, state and x[state])[0], f"out, {state}")


@pytest.mark.parametrize("aligned", [False, True], ids=["random", "aligned"])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "x".join(map(str, h)))
def test_gradients(heads, aligned):
    """Gradients of the outputs alone, with a state and without.  dg and dbeta are sums whose terms cancel in part:
    ten times 2 d is 0.36 of one rounding, and they are allowed 1.4 of it."""
    x, t = inputs(heads, aligned)
    for state in (None, "state"):
        print(f"[delta rounding] gradients {heads} aligned={aligned} state={state}", flush=True)
        args = ("q", "k", "v", "g", "beta", "dout")
        got = binding.mamba_delta_bwd(*(t[m] for m in args), initial_state=state and t[state])
        ref = delta.delta_bwd_ref(*(x[m] for m in args[:5]), heads[2] ** -0.5, x["dout"], state and x[state])
        for name in ("dq", "dk", "dv"):
            check(got[name], ref[name], name)
        for name in ("dg", "dbeta"):
            check(got[name], ref[name], name, 1.4)
