"""Calls of so many rows or heads that a launch has 2^32 threads or more: every row is done.  (A dispatch counts the
threads of a grid dimension in 32 bits; what lies past that would silently not run.)

Each case is the smallest of its kind in memory: rows of one value, heads of 8 by 8, sequences of one token.  Results
are compared on the GPU with the formula in fp32, slice by slice.
"""
import os

import pytest
import torch

from selective_state_space_47_amd import _build, binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF = torch.float32, torch.bfloat16
ROWS = (1 << 29) + 77   # 8 lanes a row: 2^32 threads and 616
SLICE = 1 << 26


@pytest.fixture(scope="module", autouse=True)
def _native():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if not os.path.exists(_build.LIB_PATH):
        _build.build()
    binding.lib()


def check(got, want, name):
    """|got - want| <= 2^-8 |want| for each bf16 value: one rounding of a few fp32 operations (2^-9, and 1e-6)."""
    for i in range(0, got.shape[0], SLICE):
        g, w = got[i:i + SLICE].float(), want(slice(i, i + SLICE))
        assert bool(((g - w).abs() <= 2.0 ** -8 * w.abs()).all()), (name, i)


def rows(n=ROWS):
    return torch.randn(n, device=DEV, dtype=BF, generator=torch.Generator(DEV).manual_seed(1))


def normed(x):
    return x * torch.rsqrt(x * x + 1e-2)


def test_gated_norm():
    y = rows()
    print("[wide] gated norm", flush=True)
    out = binding.mamba_gated_norm_fwd(y.view(-1, 1, 1), None, torch.full((1,), 2.0, device=DEV), eps=1e-2)
    check(out.view(-1), lambda s: 2.0 * normed(y[s].float()), "out")


def test_gated_norm_of_a_weight_per_group():
    """Units are rows of one group: the groups are the grid's y."""
    y = rows(2 * ROWS)
    w = torch.tensor([[2.0], [-3.0]], device=DEV)
    print("[wide] gated norm, weight per group", flush=True)
    out = binding.mamba_gated_norm_fwd(y.view(-1, 2, 1), None, w, eps=1e-2)
    check(out.view(-1), lambda s: normed(y[s].float()) * w.view(-1).repeat(len(y[s]) // 2), "out")


def test_add_norm():
    x = rows()
    print("[wide] add norm", flush=True)
    out, r = binding.mamba_add_norm_fwd(x.view(-1, 1), None, torch.full((1,), 2.0, device=DEV), eps=1e-2)
    assert torch.equal(r.view(-1), x)
    check(out.view(-1), lambda s: 2.0 * normed(x[s].float()), "out")


def test_step():
    """2^24 heads and more of 8 x 8: from a state of zero, S = beta k v^T and o = scale (q . k) beta v."""
    B, H, d = (1 << 20) + 5, 16, 8
    gen = torch.Generator(DEV).manual_seed(2)
    q, k, v = (torch.rand((B, H, d), device=DEV, generator=gen) + 0.5 for _ in range(3))
    g, beta = torch.zeros((B, H), device=DEV), torch.rand((B, H), device=DEV, generator=gen) + 0.5
    state = torch.zeros((B, H, d, d), device=DEV)
    print("[wide] step", flush=True)
    out = binding.mamba_delta_update(state, q, k, v, g, beta)
    want = d ** -0.5 * (q * k).sum(-1, keepdim=True) * beta[..., None] * v
    # all terms positive: sums of 8 products in fp32
    assert bool(((out - want).abs() <= 1e-5 * want).all())
    want = (beta[..., None] * k)[..., None] * v[..., None, :]
    assert bool(((state - want).abs() <= 1e-5 * want).all())


def test_sequences_of_one_token():
    """2^20 heads and more of 1024 columns, one token each: o = scale (q . k) beta v."""
    B, H, d, dv = (1 << 17) + 3, 8, 8, 1024
    gen = torch.Generator(DEV).manual_seed(3)

    def rand(*shape):
        return (torch.rand(shape, device=DEV, generator=gen, dtype=F32) + 0.5).to(BF)
    q, k = rand(B, 1, H, d), rand(B, 1, H, d)
    v = torch.empty((B, 1, H, dv), device=DEV, dtype=BF).uniform_(0.5, 1.5, generator=gen)
    g, beta = torch.zeros((B, 1, H), device=DEV, dtype=BF), rand(B, 1, H)
    print("[wide] sequences of one token", flush=True)
    out = binding.mamba_delta_fwd(q, k, v, g, beta)
    f = d ** -0.5 * (q.float() * k.float()).sum(-1, keepdim=True) * beta.float()[..., None]
    for i in range(0, B, 1 << 14):
        o, w = out[i:i + (1 << 14)].float(), f[i:i + (1 << 14)] * v[i:i + (1 << 14)].float()
        # one rounding to bf16 and two parts of P and E
        assert bool(((o - w).abs() <= 2.0 ** -8 * w).all()), i
