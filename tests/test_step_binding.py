"""sample_tokens, paged_plan and positions on a stream of the caller's and on their tensors' device, over the stand-ins of the
paged calls' tests."""
from types import SimpleNamespace

import pytest
import torch

import test_paged_devices
import test_paged_streams

traced = test_paged_streams.traced
two_devices = test_paged_devices.two_devices


def _plan(m, **kw):
    i = torch.ones(1, dtype=torch.int32)
    return m.paged_plan(i, i, i[None], i, i, i, 16, max_tokens=4, **kw)


def _sample(m, **kw):
    return m.sample_tokens(torch.ones(1, 2, 5), torch.ones(1, 2), probs=True, **kw)


def _positions(m, **kw):
    q, c, i = test_paged_streams._inputs()
    return m.paged_kv_append(q[:, :2], q[:, :2], c, c, i[None], i, i, positions=i, axes=[0], **kw)


CALLS = [(_plan, "paged_plan", 5), (_sample, "sample_tokens", 4), (_positions, "paged_kv_append", 1)]


@pytest.mark.parametrize("call,name,made", CALLS)
def test_outputs_are_made_on_the_calls_stream(traced, monkeypatch, call, name, made):
    m, log = traced
    monkeypatch.setattr(m, "_ext", SimpleNamespace(**{name: lambda *a: log.append(("call", a[-1]))}))
    s = SimpleNamespace(name="s", cuda_stream=7, device=torch.device("cpu"))
    call(m, stream=s)
    at = [x for x in log if x[0] in ("zeros", "empty")]
    assert len(at) == made and all(where == "s" for _, where in at)
    assert [x for x in log if x[0] == "record"] == [("record", "the caller's")] * made
    assert ("call", 7) in log


@pytest.mark.parametrize("call,name,made", CALLS)
@pytest.mark.parametrize("current", [-1, 0])
def test_the_tensors_device_is_current_in_the_call(two_devices, monkeypatch, call, name, made, current):
    m, now, calls = two_devices
    monkeypatch.setattr(m, "_ext", SimpleNamespace(**{name: lambda *a: calls.append((now[0], a[-1]))}))
    now[0] = current
    call(m)
    assert calls == [(-1, 39)] and now[0] == current


@pytest.mark.parametrize("call,name,made", CALLS)
def test_a_stream_of_another_device_is_refused(two_devices, monkeypatch, call, name, made):
    m, now, calls = two_devices
    monkeypatch.setattr(m, "_ext", SimpleNamespace(**{name: lambda *a: calls.append(a)}))
    with pytest.raises(m.AsvError) as e:
        call(m, stream=SimpleNamespace(cuda_stream=7, device=torch.device("cuda", 0)))
    assert e.value.status == 2 and not calls


@pytest.mark.parametrize("rows", [-1, 2.5, "four"])
def test_rows_of_a_plan_that_are_no_number(traced, rows):
    m, _ = traced
    i = torch.ones(1, dtype=torch.int32)
    with pytest.raises(m.AsvError):
        m.paged_plan(i, i, i[None], i, i, i, 16, max_tokens=rows,
                     stream=SimpleNamespace(name="s", cuda_stream=7, device=torch.device("cpu")))


@pytest.mark.gpu
def test_append_after_the_module_was_bound_again():
    """bind() takes the entry points that it always took; positions have one of their own."""
    import ctypes as C

    import speculative_decoding_logit_gb300 as asv
    from speculative_decoding_logit_gb300 import _binding as m
    asv.build()
    L = m.library()
    m._paged_ext().bind(m.AsvError, *(C.cast(f, C.c_void_p).value for f in (L.paged_attention, L.paged_kv_append,
                                                                            L.asv_status_string, L.asv_last_cuda_error)))
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.randn(3, 1, 16, device="cuda").bfloat16()
    table, zero, indptr = torch.tensor([[1, 0]], **i32), torch.zeros(1, **i32), torch.tensor([0, 3], **i32)
    rotary = torch.randn(16, 16, device="cuda")
    caches = []
    for kw in ({}, dict(positions=torch.arange(3, **i32))):
        kc, vc = (torch.zeros(2, 8, 1, 16, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        app = asv.paged_kv_append(k, k, kc, vc, table, zero, indptr, rotary=rotary, **kw)
        assert not app.req_status.any()
        caches.append((kc, vc))
    for a, b in zip(*caches):
        assert torch.equal(a, b) and a[1, :3].any() and not a[0].any()
