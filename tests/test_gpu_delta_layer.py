"""The example of gated delta layers: training lowers its loss, and generation one token at a time from a
packed prefill's states gives the logits of the whole sequence's prefill."""
import importlib.util
import os

import pytest
import torch

from selective_state_space_47_amd import _build, binding

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "delta_layer.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if not os.path.exists(_build.LIB_PATH):
        _build.build()
    binding.lib()
    spec = importlib.util.spec_from_file_location("delta_layer_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_trains_and_generates(example):
    print("[delta layer] 12 steps, 128 tokens", flush=True)
    losses, worst = example.main(["--steps", "12", "--tokens", "128"])
    assert losses[-1] < losses[0] - 0.05
    # both paths round every stored tensor of two layers to bf16 (2^-9 each, about ten of them in a row),
    # and round them apart where the chunked and the recurrent form differ in the last bit
    assert worst <= 2.0 ** -9 * 10


def test_gradients_equal_differences(example):
    """The whole layer's gradient against differences of the loss, along the gradient itself (where the
    difference is largest against bf16 rounding)."""
    model = example.Model(layers=1)
    data = example.sequences([64, 40, 24], 64, 3, "cuda:0")
    before = {n: t.clone() for n, t in model.layers[0].w.items()}
    model.train(*data, rate=1.0)
    grad = {n: before[n] - t for n, t in model.layers[0].w.items()}
    size = sum(float(d.norm() ** 2) for d in grad.values())
    step = 0.02 / size ** 0.5
    ends = []
    for sign in (1, -1):
        for n in before:
            model.layers[0].w[n] = before[n] + sign * step * grad[n]
        logits, _, _ = model.prefill(data[0], data[2])
        ends.append(float(torch.nn.functional.cross_entropy(logits.double(), data[1])))
    want = (ends[0] - ends[1]) / (2 * step)
    print(f"[delta layer] directional derivative {want:.4f}, gradient {size:.4f}", flush=True)
    # 128 tokens' losses of bf16 logits (2^-9 of about 10, averaged) over a step of 0.02 along the gradient
    assert abs(want - size) <= 0.1 * size
