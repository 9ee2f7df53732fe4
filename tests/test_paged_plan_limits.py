"""paged_plan from several host threads, with pools of almost 2^31 pages, and where an ended request's table holds what is no
page."""
import threading

import pytest
import torch

import test_paged_refusals as host
from test_paged_plan import State

m = host.m


@pytest.mark.gpu
def test_host_threads_plan_at_once(m):
    """Batches whose sums need more shared memory than a launch has by default, of different sizes."""
    failed, ready = [], threading.Barrier(4)

    def steps(B):
        i32 = dict(dtype=torch.int32, device="cuda")
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            one, held = torch.ones(B, **i32), torch.zeros(B, **i32)
            table, free, count = torch.full((B, 1), -1, **i32), torch.arange(B, **i32), torch.tensor([B], **i32)
            out = m.paged_plan(held.clone(), one, table, held, free, count, 8, max_tokens=B)
            s.synchronize()
            ready.wait()
            try:
                for _ in range(2000):
                    m.paged_plan(one, one, table, held, free, count, 8, out=out, stream=s)
            except m.AsvError as e:
                failed.append((B, str(e)))
            s.synchronize()
            assert held.tolist() == [1] * B and int(count) == 0
            assert out.positions.tolist() == [1] * B and not out.req_status.any()

    threads = [threading.Thread(target=steps, args=(B,)) for B in (4200, 16384, 5000, 16000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
