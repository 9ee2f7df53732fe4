"""The numbers of light tokens: log-probabilities of tokens whose weight is next to the sums' unit of 2^-44, and entries of
distributions as far down as fp32 holds them."""
import math

import numpy as np
import pytest
import torch

import test_paged_refusals as host
from sample_util import MASS, logprob_bound

m = host.m
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [(1, 8), (90, 1)])
@pytest.mark.parametrize("V,gap", [(151936, 24.25), (151936, 20.25), (1 << 19, 29.5), (300, 28.0), (5003, 26.0)])
@pytest.mark.parametrize("T", [1.0, 0.25])
def test_log_probabilities_of_light_tokens(m, dtype, rows, V, gap, T):
    """One heavy entry behind (and among) light ones, u within the light ones' mass before it.  Which of them it falls into is
    too near to tell; the number is that of the token returned."""
    B, n = rows
    x = torch.full((V,), -gap * T).to(dtype)
    x[V - 1] = 0.0
    y = x.double().numpy() / T
    for kw in (dict(), dict(top_k=5), dict(top_k=200), dict(min_p=1e-13)):
        kept = np.arange(V)
        if kw.get("top_k", V) < V:
            kept = np.append(kept[:kw["top_k"] - 1], V - 1)
        light = (len(kept) - 1) * math.exp(-gap)
        u = (light * (torch.arange(B * n).view(B, n) + 1.0) / (2.0 * B * n + 2)).float()
        got = m.sample_tokens(x.cuda().expand(B, n, V), u.cuda(), temperature=T, probs=n > 1, **kw)
        assert not got.req_status.any()
        have = got.tokens.cpu().long().numpy().ravel()
        assert np.isin(have, kept).all() and (have < V - 1).all()
        lp = y[have] - math.log1p(light)
        logs = got.logprobs.cpu().double().numpy().ravel()
        assert (np.abs(logs - lp) <= logprob_bound(lp)).all(), (kw, logs[:3], lp[:3])
        if n > 1:
            p = got.probs.cpu().double().numpy().reshape(-1, V)[np.arange(B * n), have]
            assert (np.abs(np.log(p) - logs) <= MASS + logprob_bound(lp)).all(), (kw, p[:3], logs[:3])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 90])
@pytest.mark.parametrize("T,top", [(1.0, 10.3), (0.75, 10.3), (3.0, -200.7), (0.0075, 0.103), (1.0, 1e-3)])
def test_distributions_far_below_the_maximum(m, dtype, rows, T, top):
    """Entries down to 2^-125 of the maximum, each to 2^-18 of itself: the mass, 0.75 2^-18 (sample_util); ex2, 2^-22; the mass in
    fp32 and its reciprocal, two products and a sum, 5 * 2^-24.  The exponents are sums of two floats, off by 2^-40."""
    V = 7001
    x = (top - T * 86.5 * torch.rand(V, generator=torch.Generator().manual_seed(7))).to(dtype)
    x[4321] = top
    got = m.sample_tokens(x.cuda().expand(rows, 1, V), torch.full((rows, 1), 0.5, device="cuda"), temperature=T, probs=True)
    y, T = x.double().numpy(), float(np.float32(T))
    w = np.exp((y - y.max()) / T)
    want = w / math.fsum(w)
    have = got.probs[:, 0].double().cpu().numpy()
    bound = 2.0 ** -18 * want + 2.0 ** -149
    worst = (np.abs(have - want) / bound).max()
    assert worst <= 1, (worst, np.log2(want[(np.abs(have - want) / bound).argmax() % V]))
