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
    calls, failed = [], []
    for B in (4200, 16384, 5000, 16000):
        i32 = dict(dtype=torch.int32, device="cuda")
        one, held = torch.ones(B, **i32), torch.zeros(B, **i32)
        table, free, count = torch.full((B, 1), -1, **i32), torch.arange(B, **i32), torch.tensor([B], **i32)
        out = m.paged_plan(held.clone(), one, table, held, free, count, 8, max_tokens=B)
        calls.append((one, table, held, free, count, out, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def steps(one, table, held, free, count, out, s):
        try:
            for _ in range(2000):
                m.paged_plan(one, one, table, held, free, count, 8, out=out, stream=s)
        except m.AsvError as e:
            failed.append((one.shape[0], str(e)))

    threads = [threading.Thread(target=steps, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for one, _, held, _, count, out, _ in calls:
        assert torch.equal(held, one) and int(count) == 0
        assert torch.equal(out.positions, one) and not out.req_status.any()
