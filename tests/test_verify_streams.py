"""The verification calls on a stream of the caller's: outputs and a new workspace (zero-filled) belong to that stream."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

NAMES = ["asymspec_verify", "asymspec_verify_sweep", "asymspec_sci_verify", "rapid_verify", "sci_verify"]


def _call(m, name, device, **kw):
    g = torch.Generator().manual_seed(4)
    a, b, t = (torch.randn(3, 3, 4096, generator=g).to(device) for _ in range(3))
    ids = torch.randint(0, 4096, (3, 2), generator=g).to(torch.int32).to(device)
    r = torch.full((3,), 0.6, dtype=torch.float64, device=device)
    p = b.softmax(-1)   # (here: the inputs are there before the call)
    return {"asymspec_verify": lambda: m.asymspec_verify(a, b, t, ids, **kw),
            "asymspec_verify_sweep": lambda: m.asymspec_verify_sweep(a, b, t, ids, [0.5, 1.0], [0.3, 0.5], **kw),
            "asymspec_sci_verify": lambda: m.asymspec_sci_verify(a, b, t, ids, 1.0, 0.5, r, **kw),
            "rapid_verify": lambda: m.rapid_verify(a, p, ids, **kw),
            "sci_verify": lambda: m.sci_verify(a, t, ids, r, **kw)}[name]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_and_workspace_are_made_on_the_calls_stream(monkeypatch, name):
    from speculative_decoding_logit_gb300 import _binding as m
    log, current = [], ["the caller's"]

    @contextlib.contextmanager
    def stream_context(s):
        current.append(s.name)
        yield
        current.pop()

    def noting(make):
        return lambda *a, **kw: log.append((make.__name__, current[-1])) or make(*a, **kw)

    class Library:
        def __getattr__(self, entry):
            return lambda *a: log.append((entry, a[-1])) or 0

    s = SimpleNamespace(name="s", cuda_stream=7, device=torch.device("cpu"))
    call = None
    monkeypatch.setattr(m, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    monkeypatch.setattr(m, "library", lambda: Library())
    monkeypatch.setattr(m, "_ws_cache", {})
    call = _call(m, name, "cpu", stream=s)
    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: SimpleNamespace(name=current[-1], cuda_stream=1))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)
    monkeypatch.setattr(torch, "zeros", noting(torch.zeros))
    monkeypatch.setattr(torch, "empty", noting(torch.empty))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.append(("record", s.name)))
    out = call()
    outputs = [x for x in vars(out).values() if isinstance(x, torch.Tensor)]
    made = [x for x in log if x[0] in ("zeros", "empty")]
    assert len(made) == len(outputs) + 1 and all(where == "s" for _, where in made)
    assert [x for x in log if x[0] == "record"] == [("record", "the caller's")] * len(outputs)
    assert any(handle == 7 for entry, handle in log if "verify" in entry)


def test_a_workspace_made_while_capturing_is_not_kept(monkeypatch):
    """Its zero-fill is the graph's: a later call would find it as the last replay's memory was left."""
    from speculative_decoding_logit_gb300 import _binding as m
    monkeypatch.setattr(m, "_ws_cache", {})
    capturing = [True]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    m._workspace(torch.device("cpu"), 7, 100)
    assert not m._ws_cache
    capturing[0] = False
    ws = m._workspace(torch.device("cpu"), 7, 100)
    assert m._workspace(torch.device("cpu"), 7, 200) is ws


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_a_new_workspace_is_zero_before_the_call(name):
    """The first call on a stream, the current one busy for a while: a workspace of memory that held something."""
    import speculative_decoding_logit_gb300 as asv
    asv.build()
    ref = _call(asv, name, "cuda")()
    s = torch.cuda.Stream()
    call = _call(asv, name, "cuda", stream=s)
    junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in (4096, 1 << 16, 1 << 20)]
    del junk
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    got = call()
    s.synchronize()
    torch.cuda.synchronize()
    for x, y in zip(vars(got).values(), vars(ref).values()):
        assert torch.equal(x, y)
