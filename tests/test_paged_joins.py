"""Items whose parts several CTAs file: an infinite value reaches its column alone, whichever part has it and however
many parts there are."""
import math

import pytest
import torch

from paged_long import LongBatch, Plan, attention64_wide

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def asv():
    import speculative_decoding_logit_gb300 as m
    m.build()
    return m


@pytest.mark.parametrize("group,q_len", [(1, 1), (4, 1), (8, 1), (8, 4), (5, 20), (8, 40)])
@pytest.mark.parametrize("tiles", [2, 3, 4, 5, 17, 18])
@pytest.mark.parametrize("dim", [64, 128])
def test_an_infinite_value_in_any_part(asv, group, q_len, tiles, dim):
    past = tiles * 128 - 60
    b = LongBatch([q_len], [past], heads=(group, 1), dim=dim, seed=tiles * dim + q_len)
    plan = Plan(b)
    assert all(y - x == 1 for *_, x, y, _ in plan.all())   # a part to every key tile
    v = b.v[0].clone()
    for part in sorted({0, 1, tiles // 2, tiles - 1}):
        # a position that every token attends to
        b.v[0] = v.clone()
        b.v[0][min(part * 128 + 3, past), 0, 5] = math.inf
        b.fill()
        want = attention64_wide(b)[0]
        got = asv.paged_attention(*b.args())
        assert not got.req_status.any()
        out = got.out.double()
        assert bool((out[:, :, 5] == math.inf).all()), f"part {part} of {tiles}"
        keep = [d for d in range(dim) if d != 5]
        assert bool(((out - want[0]).abs() <= want[2])[..., keep].all())
        assert bool(((got.lse.double() - want[1]).abs() <= want[3]).all())
