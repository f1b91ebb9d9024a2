"""Gradients of window attention with many sinks: sinks of every length up to all keys, long stretches of the queries that
see only them, and batches whose sinks' tiles go through all their queries.  Bounds as in test_gpu_window (2e-5 of the norm
with fp32 storage, 2^-8 with bf16)."""
import numpy as np
import pytest
import torch

from selective_state_space_47_amd import binding

from .test_gpu_window import BF, DEV, F32, GRADS, IO, _native, bwd, case, check, fwd, ids, refs, terms  # noqa: F401

pytestmark = pytest.mark.gpu


def reference(q, k, v, dout, window, sinks):
    """One layout of equally long sequences (B, L, H, d), in fp64, a query head at a time: out and the gradients."""
    B, L, Hq, d = q.shape
    rep = Hq // k.shape[2]
    t = torch.arange(L, device=DEV)
    see = (t[None] <= t[:, None]) & ((t[:, None] - t[None] < window) | (t[None] < sinks))
    out, dq = (torch.zeros(B, L, Hq, d, device=DEV, dtype=torch.float64) for _ in range(2))
    dk, dv = (torch.zeros(*k.shape, device=DEV, dtype=torch.float64) for _ in range(2))
    for b in range(B):
        for h in range(Hq):
            Q, K, V, dO = (a[b, :, i].double() for a, i in ((q, h), (k, h // rep), (v, h // rep), (dout, h)))
            P = torch.softmax((d ** -0.5 * (Q @ K.t())).masked_fill(~see, float("-inf")), 1)
            dP = dO @ V.t()
            dS = P * (dP - (P * dP).sum(1, keepdim=True)) * d ** -0.5
            out[b, :, h], dq[b, :, h] = P @ V, dS @ K
            dk[b, :, h // rep] += dS.t() @ Q
            dv[b, :, h // rep] += P.t() @ dO
    return out, dict(dq=dq, dk=dk, dv=dv)


def inputs(B, L, Hq, Hk, d, io):
    gen = torch.Generator(device=DEV).manual_seed(L + Hq)
    return [torch.randn(B, L, h, d, generator=gen, device=DEV).to(io) for h in (Hq, Hk, Hk, Hq)]


def compare(got, want, io):
    for name in want:
        off = float((got[name].double() - want[name]).norm() / want[name].norm())
        print(f"[window sinks] {name}: {off:.2e}", flush=True)
        assert off <= (2e-5 if io == F32 else 2.0 ** -8), name


# (batch, tokens, q heads, kv heads, dim, window, sinks): as many sinks as keys, one less, more; sinks that are many
# workgroups by themselves; stretches of a few queries and of 1024
SHAPES = [(1, 700, 4, 2, 64, 20, 700), (2, 333, 2, 1, 40, 1, 332), (1, 900, 2, 1, 128, 10, 1 << 40), (2, 200, 3, 3, 72, 64, 201),
          (1, 1100, 8, 8, 64, 50, 800), (3, 520, 16, 16, 24, 9, 70), (1, 450, 5, 1, 64, 100, 130), (1, 8192, 16, 1, 128, 300, 2048)]


@IO
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_gradients(shape, io):
    B, L, Hq, Hk, d, window, sinks = shape
    print(f"[window sinks] {shape} {io}", flush=True)
    q, k, v, dout = inputs(B, L, Hq, Hk, d, io)
    out, lse = binding.mamba_window_attn_fwd(q, k, v, window, sinks, return_lse=True)
    got = binding.mamba_window_attn_bwd(q, k, v, out, lse, dout, window, sinks)
    want, grads = reference(q, k, v, dout, window, sinks)
    compare(dict(got, out=out), dict(grads, out=want), io)


@IO
def test_many_short_sequences(io):
    """2000 packed sequences of 64 tokens, each with up to 1000 sinks of which it has 64: sums of stretches for every
    sequence's 63 tiles of sinks would be 8 GB."""
    B, L, Hq, Hk, d, window, sinks = 2000, 64, 8, 1, 64, 7, 1000
    print(f"[window sinks packed] {io}", flush=True)
    dims = binding.mamba_window_dims(B, B * L, B * L, Hq, Hk, d, 0, 0, 0, window, sinks, int(io == BF), 0)
    assert binding.mamba_window_attn_bwd_workspace_bytes(dims, True) < 1 << 29
    q, k, v, dout = inputs(B, L, Hq, Hk, d, io)
    off = torch.arange(0, (B + 1) * L, L, device=DEV)
    flat = [a.flatten(0, 1) for a in (q, k, v, dout)]
    out, lse = binding.mamba_window_attn_fwd(*flat[:3], window, sinks, seq_offsets=off, return_lse=True)
    got = binding.mamba_window_attn_bwd(*flat[:3], out, lse, flat[3], window, sinks, seq_offsets=off)
    some = [0, 1, 999, 1999]
    want, grads = reference(*(a[some] for a in (q, k, v, dout)), window, sinks)
    compare({n: a.unflatten(0, (B, L))[some] for n, a in dict(got, out=out).items()}, dict(grads, out=want), io)


@IO
@pytest.mark.parametrize("shape", [(2, 150, 500, 4, 2, 64, 20, 500), (1, 300, 700, 16, 16, 24, 33, 400), (2, 400, 250, 2, 1, 40, 9, 250),
                                   (1, 500, 320, 32, 32, 16, 50, 319), (1, 200, 200, 3, 1, 64, 200, 50)], ids=ids)
@pytest.mark.parametrize("scale", [None, 0.0])
def test_other_lengths(shape, scale, io):
    """Earlier keys, and queries that see none, with as many sinks as keys and with sinks that are many workgroups; and a
    scale of zero, whose weights are all the same."""
    B, n, m, Hq, Hk, d, window, sinks = shape
    x, t = case(sum(shape[:6]), B, n, m, Hq, Hk, d, io)
    print(f"[window sinks] {shape} {scale} {io}", flush=True)
    out, lse = fwd(t, window, sinks, scale=scale)
    got = bwd(t, out, lse, window, sinks, scale=scale)
    factor = d ** -0.5 if scale is None else scale
    want = [np.stack(a) for a in zip(*(refs(x, b, window, sinks, factor) for b in range(B)))]
    size = [terms(x, b, window, sinks, factor) for b in range(B)]
    check(out, want[0], "out", io)
    for name, w in zip(GRADS, want[2:]):
        check(got[name], w, name, io, terms=None if name == "dv" else np.stack([a[name] for a in size]))


@IO
def test_packed_lengths_with_many_sinks(io):
    """Sequences of different lengths, empty ones among them, with earlier keys, whose sinks are many workgroups."""
    lengths, past, H, d, window, sinks = [130, 0, 1, 260, 65], 40, 32, 16, 11, 200
    off, koff = np.cumsum([0] + lengths), np.cumsum([0] + [a + past for a in lengths])
    x, t = case(77, 1, int(off[-1]), int(koff[-1]), H, H, d, io)
    t = {a: b[0] for a, b in t.items()}
    kw = dict(seq_offsets=torch.from_numpy(off).to(DEV), kv_offsets=torch.from_numpy(koff).to(DEV))
    out, lse = fwd(t, window, sinks, **kw)
    got = bwd(t, out, lse, window, sinks, **kw)
    want, size = [], []
    for s in range(len(lengths)):
        one = dict(q=x["q"][:, off[s]:off[s + 1]], dout=x["dout"][:, off[s]:off[s + 1]],
                   k=x["k"][:, koff[s]:koff[s + 1]], v=x["v"][:, koff[s]:koff[s + 1]])
        want.append(refs(one, 0, window, sinks, d ** -0.5))
        size.append(terms(one, 0, window, sinks, d ** -0.5))
    want = [np.concatenate(a) for a in zip(*want)]
    check(out, want[0], "out", io)
    for name, w in zip(GRADS, want[2:]):
        check(got[name], w, name, io, terms=None if name == "dv" else np.concatenate([a[name] for a in size]))
