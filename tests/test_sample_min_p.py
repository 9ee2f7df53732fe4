"""min-p next to 1, where weights next to it are told apart by 2^-29 at most: the same entries are kept however a row is cut up,
and those that 64 bits give the weight of the largest are."""
import pytest
import torch

import test_paged_refusals as host
from sample_util import probs_bound

m = host.m
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 90])
@pytest.mark.parametrize("V", [7, 300, 5003, 30011])
@pytest.mark.parametrize("scale,T", [(1e-40, 1.0), (1e-20, 1e-3), (1.0, 1e18), (300.0, 1.5e19)])
@pytest.mark.parametrize("least", [1.0, 0.99999994])
def test_weights_that_64_bits_do_not_tell_from_the_largest(m, dtype, rows, V, scale, T, least):
    g = torch.Generator().manual_seed(V)
    x = (scale * torch.randn(V, generator=g)).to(dtype)
    x[::3] -= 50 * T                       # and others that are far from it
    one = torch.ones(V)
    one[::3] = 0
    want = (one / one.sum()).double()
    u = ((torch.arange(rows) + 0.5) / rows).view(rows, 1)
    at = torch.searchsorted(want.cumsum(0), u.flatten().double(), right=True).clamp(max=V - 1)
    sure = ((u.flatten().double() * float(one.sum())) % 1 - 0.5).abs() < 0.49
    for ctas in (0, 1, 2, 8):
        m.set_tuning(ctas, 0)
        try:
            for k in (0, V - 1):           # (the last of the order is one of those far from it)
                got = m.sample_tokens(x.cuda().expand(rows, 1, V), u.cuda(), temperature=T, top_k=k, min_p=least, probs=True)
                assert not got.req_status.any()
                assert bool(((got.probs[:, 0].double().cpu() - want).abs() <= probs_bound(want)).all()), (ctas, k)
                assert torch.equal(got.tokens.flatten().cpu()[sure], at.int()[sure]), (ctas, k)
        finally:
            m.set_tuning(0, 0)
