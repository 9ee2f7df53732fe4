"""Draws at and away from the borders of tokens, every row compared: u at the fp32 number nearest to a border, in a batch; u in
the middle of a token, a row at a time."""
import numpy as np
import pytest
import torch

import test_paged_refusals as host
from sample_util import logprob_bound, off, sample64
from test_sample import BF, F32, _logits_of

m = host.m


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["flat", "peaked", "ties"])
@pytest.mark.parametrize("V,B", [(20011, 64), (151936, 300)])
def test_every_draw_next_to_a_border(m, dtype, kind, V, B):
    """The token is one that u falls into with what the sums may be off by, 2^-29 + V 2^-44 of the mass, to both sides; where
    u is further than that from the borders, the one that it falls into."""
    x = _logits_of(1, 1, V, kind, dtype, V + 1)
    for k, p in ((0, 1.0), (0, 0.97), (50, 0.97)):
        p32 = float(np.float32(p))
        dist = sample64(x[0, 0].double().numpy(), 0.5, 1.0, k, p32, 0.0)[2]
        kept = np.flatnonzero(dist)
        upto = np.cumsum(dist[kept].astype(np.longdouble)).astype(float)
        u = upto[np.searchsorted(upto, np.random.default_rng(V).uniform(0.001, 0.999, B))].astype(np.float32)
        u = np.minimum(u, np.float32(1 - 2 ** -24))
        got = m.sample_tokens(x.expand(B, 1, V).cuda(), torch.from_numpy(u).view(B, 1).cuda(), top_k=k, top_p=p)
        assert not got.req_status.any()
        have = got.tokens.cpu().numpy().ravel()
        at = np.minimum(np.searchsorted(kept, have), len(kept) - 1)
        assert (kept[at] == have).all()
        u = u.astype(float)
        assert (u >= upto[at] - dist[have] - off(1.0, V)).all() and (u <= upto[at] + off(1.0, V)).all()
        first = np.searchsorted(upto, u - off(1.0, V), side="right")
        last = np.minimum(np.searchsorted(upto, u + off(1.0, V), side="right"), len(kept) - 1)
        assert (at == first)[first == last].all()
        lp = np.log(dist[have])
        assert (np.abs(got.logprobs.cpu().double().numpy().ravel() - lp) <= logprob_bound(lp)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [5, 1001, 32000, 151936])
@pytest.mark.parametrize("kind", ["peaked", "flat", "ties", "masked"])
def test_one_row_whose_draw_is_no_matter_of_borders(m, dtype, V, kind):
    x = _logits_of(1, 1, V, kind, dtype, V + 2)
    rng = np.random.default_rng(V)
    for T, k, p, least in ((1.0, 0, 1.0, 0.0), (0.8, 50, 0.95, 0.0), (0.9, 0, 0.9, 0.0), (1.2, 0, 1.0, 0.05), (1.0, 3000, 0.99, 0.0)):
        y, T32, p32, least32 = x[0, 0].double().numpy(), *(float(np.float32(v)) for v in (T, p, least))
        dist = sample64(y, 0.5, T32, k, p32, least32)[2]
        heavy = np.flatnonzero(dist >= min(1e-6, dist.max()))
        upto = np.cumsum(dist)
        for t in rng.choice(heavy, 3):
            u = np.float32(upto[t] - dist[t] / 2)
            token, lp, _, margin = sample64(y, float(u), T32, k, p32, least32)
            assert token == t
            got = m.sample_tokens(x.cuda(), torch.tensor([[u]], device="cuda"), temperature=T, top_k=k, top_p=p, min_p=least)
            if margin < 1:      # (a nucleus' border may be that near; the draw's is not)
                assert p < 1 and sample64(y, float(u), T32, k, 1.0, least32)[3] >= 1
                continue
            assert int(got.tokens) == t and not got.req_status.any()
            assert abs(float(got.logprobs) - lp) <= logprob_bound(lp)
