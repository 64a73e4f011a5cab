"""The build without a GPU: what it needs, and what it takes for up to date."""
import importlib.util
import os

from activation_sparse_gemm_b200 import build as rl_build


def test_the_library_needs_no_torch(monkeypatch):
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    assert rl_build.build() == rl_build.LIB
    assert os.path.exists(rl_build.LIB)
    assert rl_build.build_torch_calls() is None
