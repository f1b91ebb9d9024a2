"""Tensors that the binding's native part cannot hand to a kernel (CPU): refused with an error, whatever they are."""
import subprocess
import sys

import pytest
import torch

from selective_state_space_47_amd import binding

CODE = """
import warnings
warnings.simplefilter("ignore")
import torch
from selective_state_space_47_amd import binding
m = binding._marshal()
t = torch.nested.nested_tensor([torch.zeros(2, 3), torch.zeros(1, 3)])
assert t.layout == torch.strided
try:
    m.key(1, t)
except RuntimeError as e:
    print("refused")
try:
    binding.mamba_gated_norm_fwd(t, None, torch.ones(3))
except (RuntimeError, ValueError) as e:
    print("refused")
"""


def test_nested_tensor_is_refused():
    """It calls itself strided, but asking it for strides throws: in a process of its own, as an exception that
    leaves the C function ends the process."""
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == ["refused", "refused"]


def test_negated_view_is_refused():
    """Its memory holds the values with the other sign, which its sizes, strides and type do not tell."""
    m = binding._marshal()
    x = torch.randn(4, 1, 1, dtype=torch.complex64)
    for t in (x.conj().imag, torch._neg_view(torch.zeros(4, 1, 8))):
        assert t.is_neg()
        with pytest.raises(ValueError, match="resolve_neg"):
            m.key(1, t)
        with pytest.raises(ValueError, match="resolve_neg"):
            binding.mamba_gated_norm_fwd(t, None, torch.ones(t.shape[-1]))
        assert m.key(1, t.resolve_neg()) == m.key(1, torch.zeros(t.shape))


def test_module_built_for_another_torch_is_refused(monkeypatch):
    assert binding._marshal().torch_version == torch.__version__
    monkeypatch.setattr(binding, "_MARSHAL", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="built for torch"):
        binding._marshal()
