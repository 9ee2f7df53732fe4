"""How many CTAs a row gets where distributions are wanted goes by what the rows in hand keep of L2, not by the batch."""
import pytest
import torch

import test_paged_refusals as host

m = host.m


@pytest.mark.gpu
def test_small_rows_of_a_large_batch_are_not_cut_up(m):
    """4000 rows of 8192: 32 KB a row, and 131 MB of them.  Eight CTAs to a row took 2.8 times what one takes."""
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(4000, 1, 8192, device="cuda", generator=g)
    u = torch.rand(4000, 1, device="cuda", generator=g)
    out = m.sample_tokens(x, u, probs=True)
    times = {}
    try:
        for ctas in (0, 8) * 3:
            m.set_tuning(ctas, 0)
            for _ in range(3):
                m.sample_tokens(x, u, out=out)
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            for _ in range(10):
                m.sample_tokens(x, u, out=out)
            end.record()
            end.synchronize()
            times[ctas] = min(times.get(ctas, 1e9), start.elapsed_time(end))
    finally:
        m.set_tuning(0, 0)
    assert times[0] < 0.7 * times[8], times
