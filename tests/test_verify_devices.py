"""The verification calls run on their tensors' device, whichever is current, and take no other device's stream (over
stand-ins: the host tensors' device is -1 here)."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from test_verify_streams import NAMES, _call


@pytest.fixture
def two_devices(monkeypatch):
    from speculative_decoding_logit_gb300 import _binding as m
    now, calls = [0], []

    @contextlib.contextmanager
    def device_context(d):
        before, now[0] = now[0], -1 if d == torch.device("cpu") else d.index
        yield
        now[0] = before

    class Library:
        def __getattr__(self, entry):
            return lambda *a: "verify" in entry and calls.append(now[0]) or 0

    monkeypatch.setattr(m, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    monkeypatch.setattr(m, "library", lambda: Library())
    monkeypatch.setattr(m, "_ws_cache", {})
    monkeypatch.setattr(torch.cuda, "device", device_context)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: SimpleNamespace(cuda_stream=1))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda *a: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1, raising=False)
    return m, now, calls


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("current", [-1, 0])
def test_the_tensors_device_is_current_in_the_call(two_devices, name, current):
    m, now, calls = two_devices
    now[0] = current
    _call(m, name, "cpu")()
    assert calls == [-1] and now[0] == current


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(two_devices, name):
    m, now, calls = two_devices
    now[0] = -1
    with pytest.raises(m.AsvError) as e:
        _call(m, name, "cpu", stream=SimpleNamespace(cuda_stream=7, device=torch.device("cuda", 0)))()
    assert e.value.status == 2 and not calls


@pytest.mark.parametrize("current", [-1, 0])
def test_host_buffers_go_to_the_arenas_device(two_devices, current):
    m, now, calls = two_devices
    now[0] = current
    x, i = torch.zeros(2, 3, 64), torch.zeros(2, 3, dtype=torch.int32)
    m.asymspec_verify_host(x, x, x, i, 1.0, 0.5, torch.zeros(64, dtype=torch.uint8), i, i, x, i, m.ASV_F32)
    assert calls == [-1] and now[0] == current
