"""The build without a GPU: what it needs, and what it takes for up to date."""
import importlib.util
import os

import pytest

import activation_sparse_gemm_b200 as rl
from activation_sparse_gemm_b200 import build as rl_build


def test_the_library_needs_no_torch(monkeypatch):
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    assert rl_build.build() == rl_build.LIB
    assert os.path.exists(rl_build.LIB)
    assert rl_build.build_torch_calls() is None


def test_torch_calls_of_another_torch_are_not_taken(monkeypatch):
    """The compiled calls are bound to the torch that they were built against: another one finds none."""
    import torch
    built = rl_build.build_torch_calls()
    assert built == rl.torch_lib_path(torch.__version__) and os.path.exists(built)
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    monkeypatch.setattr(rl, "_calls", None)
    with pytest.raises(RuntimeError, match="0.0.0.*missing"):
        rl._torch_calls()
