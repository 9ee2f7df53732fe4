"""Building the binding's compiled module, with a stand-in for the compiler."""
import os
import stat

import pytest
import torch


@pytest.fixture
def b(monkeypatch, tmp_path):
    from speculative_decoding_logit_gb300 import nvcc_build
    nvcc_build.build()
    monkeypatch.setattr(nvcc_build, "TORCH_EXT", str(tmp_path / "asv_torch.so"))
    return nvcc_build


def _compiler(monkeypatch, tmp_path, works=True):
    """A compiler that notes its calls and writes its output (or fails)."""
    log = tmp_path / "calls"
    cc = tmp_path / "cc"
    cc.write_text(f"#!/bin/sh\necho x >> {log}\n" + (
        'while [ "$1" != "-o" ]; do shift; done\necho built > "$2"\n' if works else "echo no headers >&2\nexit 1\n"))
    cc.chmod(cc.stat().st_mode | stat.S_IEXEC)
    monkeypatch.setenv("CXX", str(cc))
    return lambda: len(log.read_text().split()) if log.exists() else 0


def test_the_module_is_built_anew_for_another_torch(b, monkeypatch, tmp_path):
    calls = _compiler(monkeypatch, tmp_path)
    b.build_torch_ext()
    b.build_torch_ext()
    assert calls() == 1
    monkeypatch.setattr(torch, "__version__", "99.0")
    b.build_torch_ext()
    b.build_torch_ext()
    assert calls() == 2


def test_a_module_of_another_torch_is_not_loaded(b, monkeypatch, tmp_path):
    from speculative_decoding_logit_gb300 import _binding
    _compiler(monkeypatch, tmp_path)
    b.build_torch_ext()
    monkeypatch.setattr(_binding, "_ext", None)
    monkeypatch.setattr(torch, "__version__", "99.0")
    with pytest.raises(_binding.AsvError, match="another PyTorch"):
        _binding._paged_ext()
