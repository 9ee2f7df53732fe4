"""fp16 caches: keys whose weights are small next to the largest, but many, count."""
import math

import pytest
import torch

from paged_long import LongBatch, attention64_wide, assert_requests

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def asv():
    import speculative_decoding_logit_gb300 as m
    m.build()
    return m


@pytest.mark.parametrize("q_len", [1, 40, 150])
@pytest.mark.parametrize("dim", [64, 128])
def test_many_small_weights(asv, q_len, dim):
    """One key of score 17.75, 20,000 of score 0: each of those weighs 2^-25.6 next to the first, together 4e-4, and only
    their values are not zero.  Twenty requests of eight key heads over the same pages, so that an item stays in one or two
    CTAs; the three sizes take the divided, the single and the two row tiles."""
    keys, B, H = 20000, 20, 8
    b = LongBatch([q_len], [keys - q_len], heads=(H, H), dim=dim, page=64, dtype=torch.float16, seed=1)
    b.k[0].zero_()
    b.k[0][0, :, 0] = 1.0
    b.qd.zero_()
    b.qd[..., 0] = 17.75
    b.v[0].fill_(1.0)
    b.v[0][0] = 0.0
    b.fill()
    want = attention64_wide(b, scale=1.0)[0]
    assert 3e-4 < float(want[0].max()) < 5e-4
    got = asv.paged_attention(b.qd.repeat(B, 1, 1), b.k_cache, b.v_cache, b.table.expand(B, -1), b.cache_len.repeat(B),
                              torch.arange(0, B * q_len + 1, q_len, dtype=torch.int32, device="cuda"), scale=1.0)
    assert not got.req_status.any()
    for r in range(B):
        one = asv.PagedAttentionOutput(got.out[r * q_len:(r + 1) * q_len], got.lse[r * q_len:(r + 1) * q_len], None)
        assert_requests(b, one, {0: want}, f"copy {r}: ")


def test_the_largest_weights_stay_in_range(asv):
    """Rows whose maximum rises by just less than what moves the reference (2^8): the weights are the largest that fp16 has
    to hold, times values near its largest."""
    b = LongBatch([1] * 20, [2000] * 20, heads=(8, 8), dim=64, page=64, dtype=torch.float16, seed=2)
    b.qd.zero_()
    b.qd[..., 0] = 1.0
    for r in range(20):
        b.k[r].zero_()
        b.k[r][128:, :, 0] = 7.99 * math.log(2)
        b.v[r].clamp_(-2, 2).mul_(2.0 ** 14)
    b.fill()
    got = asv.paged_attention(*b.args(), scale=1.0)
    assert_requests(b, got, attention64_wide(b, scale=1.0))
