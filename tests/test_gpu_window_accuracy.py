"""How exact window attention is with bf16 storage: each result is the fp32 one rounded once.

With x the kernel's value before its rounding, w the exact one and r(x) the distance of x to the bf16 it becomes: r changes
by at most |x - w| between x and w, so that |bf16(x) - w| <= r(w) + 2 |x - w|, value by value and in the 2-norm.  r(w) is
computed here from the exact value.  |x - w| is 2e-5 of the norm, as with fp32 storage, and 2^-17 from the two bf16 parts
that stand for P and for dS (the first leaves 2^-8 of a value at most, exactly, the second 2^-9 of that); of dq and dk also
2^-20 of the size of their terms, which sums of up to 128 products and the difference dout . v - D leave.
Value by value the sums' roundings may all have one sign: 128 2^-24 = 2^-17 of the sizes of the terms, once more.
"""
import numpy as np
import pytest
import torch

from oracle import window as ref

from .test_gpu_window import BF, GRADS, _native, bwd, case, fwd, ids, refs, terms  # noqa: F401

pytestmark = pytest.mark.gpu
FP32, PARTS = 2e-5, 2.0 ** -17


def rounded_once(got, want, name, sizes=None, more=0.0):
    """`sizes`: of each value's terms; `more`: what |x - w| has beside the above, in parts of the 2-norm of `sizes`."""
    got, want = got.double().cpu().numpy(), np.asarray(want)
    assert np.isfinite(got).all(), name
    own = torch.from_numpy(want).to(BF).double().numpy() - want
    size, off = np.linalg.norm(want), np.linalg.norm(got - want)
    bound = np.linalg.norm(own) + 2 * ((FP32 + PARTS) * size + more * np.linalg.norm(sizes))
    print(f"[window once] {name}: {off / size:.3e}, rounding {np.linalg.norm(own) / size:.3e}", flush=True)
    assert off <= bound, name
    assert (np.abs(got - want) <= np.abs(own) + 2 * (FP32 + 2 * PARTS) * sizes).all(), name


def sums_of_sizes(x, b, window, sinks, scale):
    """Sizes of the terms of out and dv: P |v| and P^T |dout|."""
    one = [x[m][b] for m in ("q", "k", "v")]
    out = ref.window_ref(one[0], one[1], np.abs(one[2]), window, sinks, scale)[0]
    return out, ref.window_ref(*one, window, sinks, scale, np.abs(x["dout"][b]))[2]


# (batch, queries, keys, q heads, kv heads, dim, window, sinks): windows inside a tile and of many, everything, sinks near
# and far, earlier keys, dims that do not fill a tile, keys' heads split among workgroups and not
SHAPES = [(2, 257, 257, 2, 1, 96, 1 << 40, 0), (1, 333, 333, 6, 2, 64, 100, 3), (1, 50, 300, 4, 2, 128, 64, 5),
          (1, 1400, 1400, 1, 1, 128, 200, 150), (2, 700, 700, 8, 2, 128, 128, 0), (16, 200, 200, 4, 4, 72, 17, 1)]


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_out_rounds_once(shape):
    B, n, m, Hq, Hk, d, window, sinks = shape
    x, t = case(sum(shape[:6]) + 1, B, n, m, Hq, Hk, d, BF)
    out, _ = fwd(t, window, sinks)
    want = np.stack([refs(x, b, window, sinks, d ** -0.5, grads=False)[0] for b in range(B)])
    rounded_once(out, want, "out", np.stack([sums_of_sizes(x, b, window, sinks, d ** -0.5)[0] for b in range(B)]))


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_gradients_round_once(shape):
    B, n, m, Hq, Hk, d, window, sinks = shape
    x, t = case(sum(shape[:6]) + 2, B, n, m, Hq, Hk, d, BF)
    scale = d ** -0.5
    out, lse = fwd(t, window, sinks)
    got = bwd(t, out, lse, window, sinks)
    want = [np.stack(a) for a in zip(*(refs(x, b, window, sinks, scale)[2:] for b in range(B)))]
    sizes = [dict(terms(x, b, window, sinks, scale), dv=sums_of_sizes(x, b, window, sinks, scale)[1]) for b in range(B)]
    for name, w in zip(GRADS, want):
        rounded_once(got[name], w, name, np.stack([a[name] for a in sizes]), 0.0 if name == "dv" else 2.0 ** -20)


@pytest.mark.parametrize("io", [torch.float32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("scale", [7.3, 41.0, -23.0])
def test_gradients_where_one_key_has_all_the_weight(scale, io):
    """Each query is one of its visible keys (of norms that differ), so that its score, hundreds or thousands, is far above
    the others: one weight is one, the others and dq and dk are zero, dv are the output gradients of the queries that
    chose the key.  lse, fp32, and its product with log2(e) are off by 2^-24 of themselves each, and so would be the
    weight; its difference from one would stand in dq and dk with the full size of dout . v, and in dv."""
    n, Hq, Hk, d, window, sinks = 150, 4, 2, 64, 40, 1
    x, t = case(9, 1, n, n, Hq, Hk, d, io)
    rng = np.random.default_rng(4)
    for i in range(n):
        for h in range(Hq):
            x["q"][0, i, h] = x["k"][0, rng.integers(max(0, i - window + 1), i + 1), h // 2] * np.sign(scale)
    t["q"] = torch.from_numpy(x["q"]).to(t["q"])
    out, lse = fwd(t, window, sinks, scale=scale)
    got = bwd(t, out, lse, window, sinks, scale=scale)
    want, sizes = refs(x, 0, window, sinks, scale)[2:], terms(x, 0, window, sinks, scale)
    assert float(lse.min()) > 20 * abs(scale)
    for name, w in zip(GRADS, want):
        off = np.linalg.norm(got[name][0].double().cpu().numpy() - w)
        # dq, dk: what sums of 128 products leave of dout . v - D; dv: sums of some of 80 gradients, and one rounding
        bound = 2.0 ** -20 * np.linalg.norm(sizes[name]) if name != "dv" else (
            FP32 * np.linalg.norm(w) if io != BF else
            np.linalg.norm(torch.from_numpy(w).to(BF).double().numpy() - w) + 2 * (FP32 + PARTS) * np.linalg.norm(w))
        print(f"[window one key] {scale} {io} {name}: {off:.3e}, bound {bound:.3e}", flush=True)
        assert off <= bound, name
