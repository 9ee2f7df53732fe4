"""A nucleus whose border, but for what little the lightest entries weigh, lies right behind some of several equal largest ones:
p of j equal ones' mass is a whole number of them.  Any weight besides (that 64 bits see) puts the next one in."""
import math

import pytest
import torch

import test_paged_refusals as host

m = host.m
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 90])
@pytest.mark.parametrize("V", [5, 517, 30011])
@pytest.mark.parametrize("equal,p", [(2, 0.5), (4, 0.25), (4, 0.75), (2000, 0.5), (3, 0.0), (2000, 0.0)])
@pytest.mark.parametrize("log_rest", [45.5, 47.0, 50.0, None])
def test_even_borders(m, dtype, rows, V, equal, p, log_rest):
    if equal >= V:
        return
    g = torch.Generator().manual_seed(V + equal)
    at = torch.randperm(V, generator=g)[:equal].sort().values
    for T, k in ((0.25, 0), (0.25, equal + 1), (1.0, min(V - 1, equal + 100)), (4.0, 0)):
        others = (k or V) - equal                         # that a top-k leaves
        # the others' weight together 2^-log_rest of all, or nothing
        rest = log_rest is not None and others > 0
        gap = math.inf if log_rest is None else T * (log_rest * math.log(2) + math.log(max(others, 1) / equal))
        x = torch.full((V,), 0.0 - gap).to(dtype)
        x[at] = 0.0
        u = torch.full((rows, 1), 0.9995)
        got = m.sample_tokens(x.cuda().expand(rows, 1, V), u.cuda(), temperature=T, top_k=k, top_p=p, probs=True)
        kept = int(p * equal) + int(rest) if p > 0 else 1    # (the first always)
        want = torch.zeros(V)
        want[at[:kept]] = 1.0 / kept
        assert not got.req_status.any()
        assert torch.equal(got.probs.cpu() > 0, (want > 0).expand(rows, 1, V)), (T, k, int((got.probs[0] > 0).sum()), kept)
        assert bool(((got.probs.cpu() - want).abs() <= 2.0 ** -20).all())
        assert bool((got.tokens == int(at[math.ceil(0.9995 * kept) - 1])).all())
