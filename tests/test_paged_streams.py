"""The paged calls on a stream of the caller's: what a call makes belongs to that stream."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from paged_util import Batch


@pytest.fixture
def traced(monkeypatch):
    """The binding over stand-ins: host tensors, a compiled module that notes its call, streams that note when they are
    current, allocations that note the stream they were made on."""
    from speculative_decoding_logit_gb300 import _binding
    log, current = [], ["the caller's"]

    @contextlib.contextmanager
    def stream_context(s):
        current.append(s.name)
        yield
        current.pop()

    def noting(make):
        return lambda *a, **kw: log.append((make.__name__, current[-1])) or make(*a, **kw)

    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: SimpleNamespace(name=current[-1], cuda_stream=1))
    monkeypatch.setattr(torch, "zeros", noting(torch.zeros))
    monkeypatch.setattr(torch, "empty", noting(torch.empty))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.append(("record", s.name)))
    monkeypatch.setattr(_binding, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)
    call = lambda *a: log.append(("call", a[-1]))
    monkeypatch.setattr(_binding, "_ext", SimpleNamespace(paged_attention=call, paged_kv_append=call))
    return _binding, log


def _inputs():
    q, c = torch.ones(2, 4, 64).bfloat16(), torch.ones(3, 16, 2, 64).bfloat16()
    i = torch.ones(1, dtype=torch.int32)
    return q, c, i


@pytest.mark.parametrize("append", [False, True])
def test_outputs_are_made_on_the_calls_stream(traced, append):
    m, log = traced
    q, c, i = _inputs()
    s = SimpleNamespace(name="s", cuda_stream=7, device=torch.device("cpu"))
    if append:
        m.paged_kv_append(q[:, :2], q[:, :2], c, c, i[None], i, i, q=q, stream=s)
    else:
        m.paged_attention(q, c, c, i[None], i, i, stream=s, workspace=q)
    made = [x for x in log if x[0] in ("zeros", "empty")]
    assert len(made) == (2 if append else 3) and all(where == "s" for _, where in made)
    # and are not reused before the caller's stream is done with them
    assert [x for x in log if x[0] == "record"] == [("record", "the caller's")] * len(made)
    assert ("call", 7) in log


def _bad_batch():
    b = Batch([2, 3, 1], [50, 60, 200], heads=(4, 2), dim=64, page=8, seed=2).fill()
    b.cache_len[1] = -1
    torch.cuda.synchronize()
    return b


@pytest.mark.gpu
def test_flags_of_a_call_on_another_stream_stay():
    """The current stream is busy for a while when a call with a bad length goes to another one."""
    import speculative_decoding_logit_gb300 as asv
    asv.build()
    b = _bad_batch()
    k, v = (x.cuda() for x in b.new_rows())
    s = torch.cuda.Stream()
    want = [0, asv.REQ_BAD_LEN, 0]
    for _ in range(3):
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        app = asv.paged_kv_append(k, v, b.k_cache, b.v_cache, b.table, b.cache_len, b.indptr, q=b.qd, stream=s)
        att = asv.paged_attention(app.q, b.k_cache, b.v_cache, b.table, b.cache_len, b.indptr, stream=s)
        s.synchronize()
        torch.cuda.synchronize()
        assert app.req_status.tolist() == want and att.req_status.tolist() == want


@pytest.mark.gpu
def test_outputs_of_a_call_on_another_stream_are_the_same():
    import speculative_decoding_logit_gb300 as asv
    asv.build()
    b = _bad_batch()
    ref = asv.paged_attention(b.qd, b.k_cache, b.v_cache, b.table, b.cache_len, b.indptr)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = asv.paged_attention(b.qd, b.k_cache, b.v_cache, b.table, b.cache_len, b.indptr, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got.out, ref.out) and torch.equal(got.lse, ref.lse) and torch.equal(got.req_status, ref.req_status)
