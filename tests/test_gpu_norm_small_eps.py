"""Gradients of the norms with an eps of zero or next to it, at counts of units that leave teams of the last
workgroup without one.  Bounds as in test_gpu_norm.py."""
import numpy as np
import pytest

from oracle import norm
from selective_state_space_47_amd import binding
from tests.test_gpu_norm import BF, F32, _native, check, draw, ids  # noqa: F401

import torch

pytestmark = pytest.mark.gpu
# one unit and more than a workgroup's, for teams of 8, 16, 32 and 64 lanes and for a workgroup of one team
SHAPES = [(1, 1, 64), (37, 1, 40), (5, 1, 128), (11, 3, 100), (9, 1, 256), (3, 2, 500), (5, 1, 700)]


@pytest.mark.parametrize("io", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("form", ["norm_first", "gate_first", "no_gate", "per_group"])
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_gated(shape, form, io):
    rng = np.random.default_rng(sum(shape))
    x, t = {}, {}
    for m in ("y", "z", "dout"):
        x[m], t[m] = draw(rng, shape, io)
    x["w"], t["w"] = draw(rng, shape[1:] if form == "per_group" else shape[2:], F32)
    if form == "no_gate":
        x["z"] = t["z"] = None
    first = form == "gate_first"
    print(f"[norm eps 0] {shape} {form} {io}", flush=True)
    out = binding.mamba_gated_norm_fwd(t["y"], t["z"], t["w"], eps=0.0, gate_first=first)
    check(out, norm.gated_norm_ref(x["y"], x["z"], x["w"], 0.0, first), "out")
    got = binding.mamba_gated_norm_bwd(t["y"], t["z"], t["w"], t["dout"], eps=0.0, gate_first=first)
    ref = norm.gated_norm_ref(x["y"], x["z"], x["w"], 0.0, first, x["dout"])
    for name in ("dy", "dz", "dweight"):
        if ref[name] is not None:
            check(got[name], ref[name], name)


@pytest.mark.parametrize("types", [(F32, F32), (BF, F32), (BF, BF)], ids=["f32", "bf16_f32", "bf16"])
@pytest.mark.parametrize("parts", ["all", "no_post", "bare"])
@pytest.mark.parametrize("shape", [(1, 64), (37, 40), (5, 128), (9, 256), (6, 500), (5, 700)], ids=ids)
def test_add(shape, parts, types):
    rng = np.random.default_rng(sum(shape))
    io, res = types
    x, t = {}, {}
    for m, dt in (("x", io), ("res", res), ("dout", io), ("dres", res)):
        x[m], t[m] = draw(rng, shape, dt)
    for m in ("w", "s", "p"):
        x[m], t[m] = draw(rng, shape[1:], F32)
    for m in {"all": (), "no_post": ("p",), "bare": ("p", "s")}[parts]:
        x[m] = t[m] = None
    print(f"[add norm eps 0] {shape} {parts} {types}", flush=True)
    got = binding.mamba_add_norm_bwd(t["x"], t["res"], t["w"], t["dout"], dresidual_out=t["dres"],
                                     scale=t["s"], post_weight=t["p"], eps=0.0)
    ref = norm.add_norm_ref(x["x"], x["res"], x["w"], x["s"], x["p"], 0.0, x["dout"], x["dres"])
    for name, v in ref.items():
        if v is not None:
            check(got[name], v, name)


def test_rows_of_zeros_with_an_eps_below_the_normal_range():
    """A row of zeros is divided by sqrt(eps) alone: its gradient is dout w / sqrt(eps), 1e20 of it, and the weight's
    gets nothing from it."""
    eps = float(np.float32(1e-40))
    rng = np.random.default_rng(3)
    (d, td), (w, tw) = draw(rng, (3, 1, 128), F32), draw(rng, (128,), F32)
    y = torch.zeros_like(td)
    print("[norm eps 1e-40]", flush=True)
    assert bool((binding.mamba_gated_norm_fwd(y, None, tw, eps=eps) == 0).all())
    got = binding.mamba_gated_norm_bwd(y, None, tw, td, eps=eps)
    check(got["dy"], d.astype(np.float64) * w / np.sqrt(eps), "dy")
    assert bool((got["dweight"] == 0).all())
