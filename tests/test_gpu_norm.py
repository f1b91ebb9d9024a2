"""GPU parity of the norms around a block (mamba_gated_norm_*, mamba_add_norm_* through the C ABI) against
their fp64 oracle (oracle.norm) on the same stored inputs.

Bounds per value, relative to max(|ref|, rms(ref) of its tensor):
  fp32: 1e-5.  Sums of up to 16384 squares are taken lane by lane and then as a tree (about 40 roundings
    of 2^-24), exponential, reciprocal and root add a few more; weight gradients add rows in the same way.
  bf16: 2^-8 (one rounding to bf16 is 2^-9 of the value).
"""
import os

import numpy as np
import pytest
import torch

from oracle import norm
from selective_state_space_47_amd import _build, binding, synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _native():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if not os.path.exists(_build.LIB_PATH):
        _build.build()
    binding.lib()


def check(got, ref, name):
    ref = np.asarray(ref)
    tol = 1e-5 if got.dtype == F32 else 2.0 ** -8
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape and np.isfinite(got).all(), name
    rms = float(np.sqrt(np.mean(ref * ref)))
    e = float(np.max(np.abs(got - ref) / np.maximum(np.abs(ref), rms))) if rms else np.abs(got).max()
    print(f"[norm] {name}: {e:.2e}", flush=True)
    assert e <= tol, name


def draw(rng, shape, io):
    x = rng.standard_normal(shape).astype(np.float32)
    x = synth.round_to_bf16(x) if io == BF else x
    return x, torch.from_numpy(x).to(DEV).to(io)


# (rows, groups, dim): every width of team, its edges, odd sizes, one row and ragged last workgroups
GATED = [(1, 1, 1), (3, 2, 7), (70, 5, 64), (33, 3, 72), (5, 4, 128), (17, 2, 200), (9, 1, 257),
         (4, 3, 513), (7, 1, 768), (2, 1, 1237), (3, 2, 2048), (2, 1, 2560), (3, 1, 5120), (2, 1, 8191),
         (2, 1, 16384)]
ids = lambda s: "x".join(map(str, s))  # noqa: E731


@pytest.mark.parametrize("io", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", GATED, ids=ids)
@pytest.mark.parametrize("form", ["norm_first", "gate_first", "no_gate"])
def test_gated_norm(shape, io, form):
    rng = np.random.default_rng(sum(shape))
    rows, G, d = shape
    gate_first = form == "gate_first"
    per_group = G > 1 and form != "no_gate"
    x, t = {}, {}
    for m in ("y", "z", "dout"):
        x[m], t[m] = draw(rng, shape, io)
    x["w"], t["w"] = draw(rng, (G, d) if per_group else (d,), F32)
    if form == "no_gate":
        x["z"] = t["z"] = None
    else:  # z as a slice of a wider row that starts at an odd element
        wide = torch.full((rows, G * d + 5), float("nan"), device=DEV, dtype=io)
        wide[:, 3:3 + G * d] = t["z"].flatten(1)
        t["z"] = wide[:, 3:3 + G * d].unflatten(1, (G, d))
    print(f"[gated norm] {shape} {io} {form}", flush=True)
    out = binding.mamba_gated_norm_fwd(t["y"], t["z"], t["w"], eps=1e-3, gate_first=gate_first)
    check(out, norm.gated_norm_ref(x["y"], x["z"], x["w"], 1e-3, gate_first), "out")
    got = binding.mamba_gated_norm_bwd(t["y"], t["z"], t["w"], t["dout"], eps=1e-3,
                                       gate_first=gate_first)
    ref = norm.gated_norm_ref(x["y"], x["z"], x["w"], 1e-3, gate_first, x["dout"])
    for name in ("dy", "dz", "dweight"):
        if ref[name] is None:
            assert got[name] is None
        else:
            check(got[name], ref[name], name)


@pytest.mark.parametrize("types", [(F32, F32), (BF, F32), (BF, BF)], ids=["f32", "bf16_f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (70, 64), (9, 130), (300, 257), (1, 768), (33, 1237),
                                   (5, 2000), (1030, 2560), (3, 4096), (2, 5120), (2, 8191), (2, 16384)],
                         ids=ids)
@pytest.mark.parametrize("parts", ["all", "no_post", "bare", "no_residual"])
def test_add_norm(shape, types, parts):
    rng = np.random.default_rng(sum(shape))
    io, res = types
    x, t = {}, {}
    for m, dt in (("x", io), ("res", res), ("dout", io), ("dres", res)):
        x[m], t[m] = draw(rng, shape, dt)
    for m in ("w", "s", "p"):
        x[m], t[m] = draw(rng, shape[1:], F32)
    for m in {"all": (), "no_post": ("p",), "bare": ("p", "s", "dres"), "no_residual": ("res",)}[parts]:
        x[m] = t[m] = None
    print(f"[add norm] {shape} {types} {parts}", flush=True)
    r_out = torch.empty(shape, dtype=res, device=DEV)
    out, r = binding.mamba_add_norm_fwd(t["x"], t["res"], t["w"], scale=t["s"], post_weight=t["p"],
                                        eps=1e-3, residual_out=r_out)
    ro, rr = norm.add_norm_ref(x["x"], x["res"], x["w"], x["s"], x["p"], 1e-3)
    check(out, ro, "out")
    check(r, rr, "residual_out")
    assert r.dtype == res
    got = binding.mamba_add_norm_bwd(t["x"], t["res"], t["w"], t["dout"], dresidual_out=t["dres"],
                                     scale=t["s"], post_weight=t["p"], eps=1e-3)
    ref = norm.add_norm_ref(x["x"], x["res"], x["w"], x["s"], x["p"], 1e-3, x["dout"], x["dres"])
    for name, v in ref.items():
        if v is None:
            assert got[name] is None
        else:
            check(got[name], v, name)


@pytest.mark.parametrize("io", [F32, BF], ids=["f32", "bf16"])
def test_rows_of_zeros_and_wide_gates(io):
    """A row of zeros has a norm of zero and a finite gradient; gates of +-100 saturate without NaN."""
    rng = np.random.default_rng(5)
    x, t = {}, {}
    for m in ("y", "z", "dout"):
        x[m], t[m] = draw(rng, (6, 2, 128), io)
    for a in (x, t):
        a["y"][2] = 0.0
        a["z"][3, 0] = 100.0
        a["z"][3, 1] = -100.0
        a["z"][4] = 0.0
    w, tw = draw(rng, (128,), F32)
    print(f"[norm zeros] {io}", flush=True)
    for gate_first in (False, True):
        out = binding.mamba_gated_norm_fwd(t["y"], t["z"], tw, gate_first=gate_first)
        check(out, norm.gated_norm_ref(x["y"], x["z"], w, 1e-5, gate_first), "out")
        assert bool((out[2] == 0).all()) and bool((out[4] == 0).all())
        if not gate_first:  # (gate first, row 4's gradient is 1 / sqrt(eps) large and drowns the rest)
            got = binding.mamba_gated_norm_bwd(t["y"], t["z"], tw, t["dout"], gate_first=gate_first)
            ref = norm.gated_norm_ref(x["y"], x["z"], w, 1e-5, gate_first, x["dout"])
            for name in ("dy", "dz", "dweight"):
                check(got[name], ref[name], name)


def test_norm_gradients_equal_differences():
    """Directional differences of the library's own fp32 forward against its gradients."""
    rng = np.random.default_rng(6)
    t = {m: draw(rng, (5, 2, 96), F32)[1] for m in ("y", "z", "dout")}
    t["w"] = draw(rng, (96,), F32)[1]
    got = binding.mamba_gated_norm_bwd(t["y"], t["z"], t["w"], t["dout"])
    print("[norm differences]", flush=True)
    for m, name in (("y", "dy"), ("z", "dz"), ("w", "dweight")):
        way = draw(rng, tuple(t[m].shape), F32)[1]
        ends = []
        for sign in (1, -1):
            u = dict(t, **{m: t[m] + sign * 2e-3 * way})
            ends.append(float((binding.mamba_gated_norm_fwd(u["y"], u["z"], u["w"]).double()
                               * t["dout"].double()).sum()))
        have = float((got[name].double() * way.double()).sum())
        # the step's square, and fp32 outputs over the step
        assert abs(have - (ends[0] - ends[1]) / 4e-3) <= 2e-3 * float(got[name].norm() * way.norm())


def test_in_place_residual_determinism_and_stream():
    """The residual stream updated in place, on another stream, twice: bitwise the same."""
    rng = np.random.default_rng(7)
    x, r = draw(rng, (40, 320), BF)[1], draw(rng, (40, 320), F32)[1]
    w, d = draw(rng, (320,), F32)[1], draw(rng, (40, 320), BF)[1]
    print("[norm in place]", flush=True)
    out, new = binding.mamba_add_norm_fwd(x, r, w)
    g = binding.mamba_add_norm_bwd(x, r, w, d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        mine = r.clone()
        o2, r2 = binding.mamba_add_norm_fwd(x, mine, w, residual_out=mine)
        g2 = binding.mamba_add_norm_bwd(x, r, w, d)
    s.synchronize()
    assert r2 is mine and torch.equal(o2, out) and torch.equal(mine, new)
    assert all(torch.equal(g[n], g2[n]) for n in ("dx", "dresidual", "dweight"))


def test_refusals():
    y = torch.zeros((4, 2, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    gn, an = binding.mamba_gated_norm_fwd, binding.mamba_add_norm_fwd
    x = torch.zeros((4, 64), device=DEV)
    bad = [lambda: gn(y, y.bfloat16(), w), lambda: gn(y, y[:3], w), lambda: gn(y, y, w[:32]),
           lambda: gn(y, y, w.bfloat16()), lambda: gn(y.transpose(1, 2), None, w),
           lambda: gn(y[0], None, w), lambda: gn(y, y, w, eps=-1.0), lambda: gn(y, y, w, eps=float("nan")),
           lambda: gn(y, y, w, out=torch.empty((4, 2, 32), device=DEV)), lambda: gn(y.cpu(), None, w),
           lambda: gn(torch.zeros((1, 1, 16385), device=DEV), None, torch.ones(16385, device=DEV)),
           lambda: binding.mamba_gated_norm_bwd(y, y, w, None),
           lambda: binding.mamba_gated_norm_bwd(y, y, w, y, workspace=torch.empty(4, device=DEV)),
           lambda: an(x, x[:2], w), lambda: an(x, x.bfloat16(), w), lambda: an(x, x.half(), w),
           lambda: an(x, x, w[:2]), lambda: an(x, x, w, scale=w.bfloat16()), lambda: an(x.t(), None, w),
           lambda: an(x, x, None), lambda: an(x[:0], None, w),
           lambda: binding.mamba_add_norm_bwd(x, x, w, None),
           lambda: binding.mamba_add_norm_bwd(x, x, w, x, dresidual_out=x.bfloat16())]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print(f"refusal {i} did not happen", flush=True)
