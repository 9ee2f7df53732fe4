"""Rows whose values lie on both sides of 0 so near to it that their bits are next to each other: -0 and 0 are one value, and the
brackets of a border are ranges of bits."""
import pytest
import torch

import test_paged_refusals as host

m = host.m
BF, F32 = torch.bfloat16, torch.float32
ULP = 2.0 ** -149


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 90])
@pytest.mark.parametrize("V", [5003, 30011])
@pytest.mark.parametrize("top", [511, 512, 4095, 4096, 1023])
@pytest.mark.parametrize("dense", [False, True])
def test_borders_next_to_zero(m, rows, V, top, dense):
    """Weights that are all the same, so the kept set's size is known; the order is by value, then by index."""
    g = torch.Generator().manual_seed(V + top)
    steps = torch.randint(-(511 if dense else 400_000), 1, (V,), generator=g)
    steps[torch.rand(V, generator=g) < 0.3] = torch.randint(0, top, (1,), generator=g)
    zero = torch.rand(V, generator=g) < 0.05
    steps[zero] = 0
    steps[V // 3] = top
    x = (steps.double() * ULP).float()
    x[zero & (torch.rand(V, generator=g) < 0.5)] = -0.0
    order = torch.sort(-steps, stable=True).indices
    u = ((torch.arange(rows) + 0.5) / rows).view(rows, 1)
    for p in (0.31, 0.34, 0.36, 0.5, 0.9):
        kept = int((torch.arange(V).double() < float(torch.tensor(p)) * V).sum())
        for kw in (dict(top_p=p), dict(top_k=kept), dict(top_p=p, min_p=0.5)):
            got = m.sample_tokens(x.cuda().expand(rows, 1, V), u.cuda(), probs=True, **kw)
            assert not got.req_status.any()
            want = torch.zeros(V, dtype=torch.bool)
            want[order[:kept]] = True
            assert torch.equal(got.probs[:, 0].cpu() > 0, want.expand(rows, V)), (kw, kept, (got.probs[0] > 0).sum())
            at = want.nonzero().flatten()
            place = u.flatten().double() * kept
            sure = (place % 1 - 0.5).abs() < 0.49
            assert torch.equal(got.tokens.flatten().cpu()[sure].long(), at[place.long().clamp(max=kept - 1)][sure])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 90])
def test_zeros_of_both_signs(m, dtype, rows):
    """They tie: the lowest index first, whatever the sign."""
    V = 20011
    x = torch.where(torch.rand(V, generator=torch.Generator().manual_seed(1)) < 0.5, 0.0, -0.0).to(dtype)
    x[::7] = -3.0
    at = (x == 0).nonzero().flatten()
    for kw, kept in ((dict(top_k=1), 1), (dict(top_k=7000), 7000), (dict(temperature=0.0), 1), (dict(min_p=0.5), len(at))):
        got = m.sample_tokens(x.cuda().expand(rows, 1, V), torch.full((rows, 1), 0.999999, device="cuda"), probs=True, **kw)
        want = torch.zeros(V, dtype=torch.bool)
        want[at[:kept]] = True
        assert torch.equal(got.probs[:, 0].cpu() > 0, want.expand(rows, V))
        assert bool((got.tokens == int(at[kept - 1])).all())
