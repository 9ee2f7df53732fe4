"""The paged calls run on their tensors' device, whichever is current, and take no other device's stream (over stand-ins: the
host tensors' device is -1 here)."""
import contextlib
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture
def two_devices(monkeypatch):
    from speculative_decoding_logit_gb300 import _binding
    now, calls = [0], []

    @contextlib.contextmanager
    def device_context(d):
        before, now[0] = now[0], -1 if d == torch.device("cpu") else d.index
        yield
        now[0] = before

    monkeypatch.setattr(torch.cuda, "device", device_context)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 40 + d, raising=False)
    monkeypatch.setattr(_binding, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "stream", contextlib.nullcontext)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda *a: None)
    call = lambda *a: calls.append((now[0], a[-1]))
    monkeypatch.setattr(_binding, "_ext", SimpleNamespace(paged_attention=call, paged_kv_append=call))
    return _binding, now, calls


def _call(m, append, **kw):
    q, c = torch.ones(2, 4, 64).bfloat16(), torch.ones(3, 16, 2, 64).bfloat16()
    i = torch.ones(1, dtype=torch.int32)
    if append:
        return m.paged_kv_append(q[:, :2], q[:, :2], c, c, i[None], i, i, q=q, **kw)
    return m.paged_attention(q, c, c, i[None], i, i, workspace=q, **kw)


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("current", [-1, 0])
def test_the_tensors_device_is_current_in_the_call(two_devices, append, current):
    m, now, calls = two_devices
    now[0] = current
    got = _call(m, append)
    assert calls == [(-1, 39)] and got.req_status.numel() == 1
    assert now[0] == current


@pytest.mark.parametrize("append", [False, True])
def test_a_stream_of_another_device_is_refused(two_devices, append):
    m, now, calls = two_devices
    s = SimpleNamespace(cuda_stream=7, device=torch.device("cuda", 0))
    with pytest.raises(m.AsvError) as e:
        _call(m, append, stream=s)
    assert e.value.status == 2 and not calls
