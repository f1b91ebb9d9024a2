"""The native part of the binding's calls (CPU): new tensors, and refusals instead of crashes."""
import pytest
import torch

from selective_state_space_47_amd import binding


@pytest.fixture(scope="module")
def m():
    return binding._marshal()


def test_empty_is_a_plain_contiguous_tensor(m):
    like = torch.nn.Parameter(torch.zeros(6, 5, dtype=torch.bfloat16))[::2]
    t = m.empty(like)
    assert type(t) is torch.Tensor and t.shape == (3, 5) and t.dtype == torch.bfloat16
    assert t.is_contiguous() and not t.requires_grad and t.device == like.device
    t = m.empty(like, "f", 2, 0, 4, 1)
    assert t.shape == (2, 0, 4, 1) and t.dtype == torch.float32
    t = m.empty(like, "b", 100)
    assert t.shape == (100,) and t.dtype == torch.uint8
    with torch.inference_mode():
        assert m.empty(like).is_inference()


@pytest.mark.parametrize("args", [(), (3,), (None, "f", 1), ("like", 1), ("like", "f", 1, 2, 3, 4, 5),
                                  ("like", "f", "x")])
def test_empty_refuses(m, args):
    args = tuple(torch.zeros(2) if a == "like" else a for a in args)
    with pytest.raises(TypeError):
        m.empty(*args)


def test_empty_of_negative_size(m):
    with pytest.raises(RuntimeError):
        m.empty(torch.zeros(2), "f", -1)


def test_key_tells_calls_apart(m):
    a = torch.zeros(4, 6)
    keys = [m.key(1, a), m.key(2, a), m.key(1, a.bfloat16()), m.key(1, a[:2]), m.key(1, a.t()), m.key(1, None),
            m.key(1, a, None), m.key(1, True), m.key(1, 1), m.key(1, "a")]
    assert len(set(keys)) == len(keys)
    assert m.key(1, a) == m.key(1, torch.ones(4, 6))
