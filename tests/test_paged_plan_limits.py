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


@pytest.mark.gpu
def test_almost_all_pages_that_32_bits_can_number_given_back(m):
    """2^31 - 1 pages held by 16,384 requests that have all ended: a thread's next page's number is past 31 bits."""
    B, width = 16384, 131072
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.arange(width, **i32) + (torch.arange(B, **i32) * width)[:, None]
    held, pool, count = torch.full((B,), width, **i32), torch.zeros(B * width - 1, **i32), torch.zeros(1, **i32)
    held[-1] -= 1
    new = torch.zeros(B, **i32)
    new[7] = 3
    plan = m.paged_plan(torch.zeros(B, **i32), new, table, held, pool, count, 16, max_tokens=2100,
                        release=torch.ones(B, dtype=torch.bool, device="cuda"))
    assert not plan.req_status.any() and int(count) == B * width - 2
    top = B * width - 2
    assert plan.slots[:4].tolist() == [top * 16, top * 16 + 1, top * 16 + 2, -1]
    for i in range(0, B * width - 1, 1 << 28):
        part = pool[i:i + (1 << 28)]
        assert bool((part == torch.arange(i, i + part.shape[0], device="cuda")).all())
    assert int(table[7, 0]) == top and int(table[-1, -1]) == B * width - 1
    table[7, 0] = table[-1, -1] = -1
    assert bool((table == -1).all())
    assert held.tolist() == [0] * 7 + [1] + [0] * (B - 8)


@pytest.mark.gpu
def test_negative_entries_among_the_pages_given_back(m):
    """They are what the table holds, so they go onto the pool, and the request that held them is flagged."""
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.tensor([[4, 5, -9], [6, -2, 7]], **i32)
    held, pool, count = torch.tensor([2, 3], **i32), torch.tensor([1, 0, 0, 0, 0, 0, 0], **i32), torch.tensor([1], **i32)
    zero = torch.zeros(2, **i32)
    plan = m.paged_plan(zero, zero, table, held, pool, count, 8, max_tokens=1,
                        release=torch.ones(2, dtype=torch.bool, device="cuda"))
    assert plan.req_status.tolist() == [0, m.REQ_BAD_PAGE] and held.tolist() == [0, 0]
    assert pool.tolist() == [1, 4, 5, 6, -2, 7, 0] and count.tolist() == [6]
    assert table.tolist() == [[-1, -1, -9], [-1, -1, -1]]


@pytest.mark.gpu
def test_a_block_table_without_dimensions_is_refused(m):
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(m.AsvError) as e:
        m.paged_plan(i, i, i[0], i, i, i, 16, max_tokens=3)
    assert e.value.status == 2
