"""Pins of the fp64 references of the gated delta rule and of the norms (CPU): hand-worked cases, and
every gradient against central finite differences of the forward."""
import numpy as np
import pytest

from oracle import delta, norm


def _diff(f, x, eps=1e-6):
    """Central differences of the scalar f() in every element of x (changed in place)."""
    d = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + eps
        up = f()
        x[i] = keep - eps
        d[i] = (up - f()) / (2 * eps)
        x[i] = keep
    return d


def test_delta_by_hand():
    """One head, dk = dv = 1: the state is a number, and three tokens are worked out by hand."""
    one = lambda *a: np.array(a, dtype=np.float64).reshape(1, 3, 1, 1)  # noqa: E731
    q, k, v = one(1, 2, 3), one(1, 1, 0.5), one(4, 1, 2)
    g, beta = np.log([[[1.0], [0.5], [0.25]]]).reshape(1, 3, 1), np.array([[[0.5], [1.0], [2.0]]])
    out, last = delta.delta_ref(q, k, v, g, beta, 10.0, np.full((1, 1, 1, 1), 2.0))
    # S: 2 -> 2 + .5 (4 - 2) = 3 -> 1.5 + (1 - 1.5) = 1 -> .25 + 2 * .5 (2 - .125) = 2.125
    assert np.allclose(out.ravel(), [30.0, 20.0, 63.75]) and np.allclose(last.ravel(), 2.125)


def test_delta_rule_overwrites_a_key():
    """beta = 1 and unit keys: the value stored last for a key is read back whole."""
    k = np.zeros((1, 3, 1, 4))
    k[0, :, 0, 2] = 1.0
    v = np.random.default_rng(0).standard_normal((1, 3, 1, 5))
    out, _ = delta.delta_ref(k, k, v, np.zeros((1, 3, 1)), np.ones((1, 3, 1)), 1.0)
    assert np.allclose(out, v)


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (2, 4)])
def test_delta_gradients_equal_differences(Hk, Hv):
    rng = np.random.default_rng(Hv)
    B, L, dk, dv = 2, 4, 3, 2
    x = dict(q=rng.standard_normal((B, L, Hk, dk)), k=rng.standard_normal((B, L, Hk, dk)) * 0.6,
             v=rng.standard_normal((B, L, Hv, dv)), g=-rng.random((B, L, Hv)),
             beta=rng.random((B, L, Hv)), state=rng.standard_normal((B, Hv, dk, dv)))
    dout, dlast = rng.standard_normal((B, L, Hv, dv)), rng.standard_normal((B, Hv, dk, dv))

    def loss():
        out, last = delta.delta_ref(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.7, x["state"])
        return (out * dout).sum() + (last * dlast).sum()

    got = delta.delta_bwd_ref(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.7, dout, x["state"],
                              dlast)
    for name, key in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"), ("dbeta", "beta"),
                      ("dinitial_state", "state")):
        want = _diff(loss, x[key])
        # central differences: eps^2 of the third derivative, and 2^-52 / eps of the loss
        assert np.abs(got[name] - want).max() <= 1e-7 * max(1.0, np.abs(want).max()), name


@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("per_group", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_gated_norm_gradients_equal_differences(gate_first, per_group, gate):
    rng = np.random.default_rng(3)
    y, z = rng.standard_normal((3, 2, 4)), rng.standard_normal((3, 2, 4)) if gate else None
    w, d = rng.standard_normal((2, 4) if per_group else 4), rng.standard_normal((3, 2, 4))
    loss = lambda: (norm.gated_norm_ref(y, z, w, 1e-3, gate_first) * d).sum()  # noqa: E731
    got = norm.gated_norm_ref(y, z, w, 1e-3, gate_first, d)
    for name, t in (("dy", y), ("dz", z), ("dweight", w)):
        if t is not None:
            assert np.abs(got[name] - _diff(loss, t)).max() <= 1e-7, name


@pytest.mark.parametrize("residual,scale,post", [(True, True, True), (True, False, False),
                                                 (False, True, False), (False, False, True)])
def test_add_norm_gradients_equal_differences(residual, scale, post):
    rng = np.random.default_rng(4)
    x, q = rng.standard_normal((3, 5)), rng.standard_normal((3, 5)) if residual else None
    w, s, p = rng.standard_normal(5), rng.standard_normal(5), rng.standard_normal(5)
    s, p = s if scale else None, p if post else None
    d, dr = rng.standard_normal((3, 5)), rng.standard_normal((3, 5))

    def loss():
        out, r = norm.add_norm_ref(x, q, w, s, p, 1e-3)
        return (out * d).sum() + (r * dr).sum()

    got = norm.add_norm_ref(x, q, w, s, p, 1e-3, d, dr)
    for name, t in (("dx", x), ("dresidual", q), ("dweight", w), ("dscale", s), ("dpost_weight", p)):
        if t is not None:
            assert np.abs(got[name] - _diff(loss, t)).max() <= 1e-7, name
        else:
            assert got[name] is None


def test_norms_by_hand():
    y = np.array([[[3.0, 4.0]]])
    out = norm.gated_norm_ref(y, None, np.array([1.0, 2.0]), 0.0, False)
    assert np.allclose(out, [[[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]]])
    out, r = norm.add_norm_ref(np.array([[1.0, 2.0]]), np.array([[2.0, 0.0]]), np.ones(2),
                               np.array([1.0, 2.0]), None, 0.0)
    assert np.allclose(r, [[3, 4]]) and np.allclose(out, [[3 / np.sqrt(12.5), 4 / np.sqrt(12.5)]])
