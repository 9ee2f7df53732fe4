"""Draws from the whole row where its logits are many temperatures away from 0, on both sides of what the fast sums' finer
form takes ((max / T) log2(e) of 4000) and of what fast sums take at all (2^20)."""
import math

import numpy as np
import pytest
import torch

import test_paged_refusals as host
from sample_util import logprob_bound, off

m = host.m
BF, F32 = torch.bfloat16, torch.float32


def _row(kind, V, value, dtype):
    g = torch.Generator().manual_seed(V)
    x = torch.full((V,), value, dtype=dtype)
    if kind == "tied":           # a third at the maximum, the others steps of the type below it
        step = abs(value) * torch.finfo(dtype).eps
        x[torch.rand(V, generator=g) < 2 / 3] = value - step * 2
    elif kind == "spread":       # a few hundred neighbouring values
        x += (value * torch.finfo(dtype).eps * torch.randint(0, 300, (V,), generator=g)).to(dtype)
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [(1, 1), (1, 16), (90, 1)])
@pytest.mark.parametrize("far", [3999.0, 4001.0, 1e5, 1.04e6, 2.0 ** 20, 3e6])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("kind", ["equal", "tied", "spread"])
def test_draws_from_rows_far_from_zero(m, dtype, rows, far, sign, kind):
    B, n = rows
    for V in (30011, 151936):
        T = float(np.float32(64 / math.log(2) / far))
        x = _row(kind, V, sign * 64.0, dtype)
        u = torch.arange(B * n).view(B, n) / (B * n) + 0.3 / (B * n)
        got = m.sample_tokens(x.cuda().expand(B, n, V), u.cuda(), temperature=T)
        assert not got.req_status.any()
        y = x.double().numpy()
        w = np.exp((y - y.max()) / T)
        upto = np.cumsum(w.astype(np.longdouble))
        at = u.double().numpy().ravel() * upto[-1]
        want = np.searchsorted(upto, at, side="right")
        # (how near the draw's borders are, in what the sums may be off by)
        before = upto[want] - w[want]
        near = np.minimum(upto[want] - at, np.where(before > 0, at - before, np.inf)) / off(float(upto[-1]), V)
        sure = near >= 1
        assert sure.mean() >= 0.9
        have = got.tokens.cpu().numpy().ravel()
        assert (have == want)[sure].all(), (T, V, have[sure & (have != want)], want[sure & (have != want)])
        lp = np.log(w[have] / float(upto[-1]))
        assert (np.abs(got.logprobs.cpu().double().numpy().ravel() - lp) <= logprob_bound(lp)).all()
