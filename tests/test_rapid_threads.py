"""rapid_verify_ex from several host threads, vocabularies that need different amounts of shared memory: each gets what it
gets alone."""
import ctypes as C
import threading

import pytest
import torch

import speculative_decoding_logit_gb300 as asv
from speculative_decoding_logit_gb300 import _binding as m


@pytest.mark.gpu
def test_host_threads_verify_at_once():
    asv.build()
    calls, failed = [], []
    option = m._RapidOptionsC(0)
    asv.set_tuning(1, 0)
    try:
        for V in (20000, 72000, 100000, 151936):
            g = torch.Generator("cuda").manual_seed(V)
            z = torch.randn(1, 2, V, device="cuda", generator=g)
            q = torch.randn(1, 2, V, device="cuda", generator=g).softmax(-1)
            ids = torch.randint(0, V, (1, 1), dtype=torch.int32, device="cuda", generator=g)
            out = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (1, 2, 1)]
            work = torch.zeros(asv.workspace_bytes(m.ASV_MODE_RAPID, 1, 1, V, m.ASV_F32), dtype=torch.uint8, device="cuda")
            s = torch.cuda.Stream()
            calls.append((z, q, ids, out, work, s, (
                z.data_ptr(), q.data_ptr(), ids.data_ptr(), 1, 1, V, 1.0, 10.0, 0.1, 1234, 0, C.byref(option),
                *(t.data_ptr() for t in out), work.data_ptr(), work.numel(), s.cuda_stream)))
        torch.cuda.synchronize()
        call, together = m.library().rapid_verify_ex, threading.Barrier(len(calls))

        def steps(args):
            together.wait(60)
            failed.extend(x for x in [call(*args) for _ in range(2000)] if x)

        threads = [threading.Thread(target=steps, args=(c[-1],)) for c in calls]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not failed
        for z, q, ids, out, _, _, _ in calls:
            want = asv.rapid_verify(z, q, ids)
            for a, b in zip(out, (want.accept_len, want.tokens, want.req_status)):
                assert torch.equal(a.view(-1), b.view(-1))
    finally:
        asv.set_tuning(0, 0)
