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


def test_the_library_is_built_without_the_module(b, monkeypatch, tmp_path):
    """The verification needs no compiled module: where the host compiler fails, build() says so and the paged calls
    refuse, with a module of older sources out of the way."""
    from speculative_decoding_logit_gb300 import _binding
    _compiler(monkeypatch, tmp_path)
    b.build_torch_ext()
    os.utime(b.TORCH_EXT, (1, 1))   # older than its sources
    _compiler(monkeypatch, tmp_path, works=False)
    with pytest.warns(RuntimeWarning, match="no headers"):
        assert b.build() == b.LIB
    assert os.path.exists(b.LIB) and not os.path.exists(b.TORCH_EXT)
    monkeypatch.setattr(_binding, "_ext", None)
    with pytest.raises(_binding.AsvError, match="not built"):
        _binding._paged_ext()
    assert _binding.workspace_bytes(0, 1, 2, 4096, 0) > 0
    with pytest.raises(RuntimeError, match="no headers"):   # asked for by itself it is an error
        b.build_torch_ext()
