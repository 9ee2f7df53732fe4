"""paged_kv_append with positions of several axes: each pair turned by the position on its own axis against 64 bits
(paged_util.rotate64's bound: two products and a sum in fp32, one rounding), slots by cache_len as ever, and the refusals."""
import ctypes as C

import pytest
import torch

import test_paged_refusals as host
from paged_util import Batch, assert_within, rotate64, rotation_table

NULL, SHAPE, ALIGN, DTYPE, PARAM = 1, 2, 3, 4, 5
m = host.m


# ------------------------------------------------------------------ refusals, on the host

def _append(m, rot=None, at=None, **kw):
    ref = lambda x: None if x is None else C.addressof(x)
    cache, batch = host._cache(m), host._batch(m)
    return m.library().paged_kv_append_ex(C.addressof(cache), C.addressof(batch), None, None, None, None, 4, ref(rot),
                                          ref(at), None, None)


def test_positions_are_checked(m):
    rot = m._RotaryC(None, 64, 10, 0)
    ok = bytes([0, 1, 2, 2] * 8)
    assert _append(m, at=m._PositionsC(None, 1, 0, None)) == PARAM            # no rotation
    for n in (0, -1, 9):
        assert _append(m, rot, m._PositionsC(None, n, 0, None)) == PARAM
    assert _append(m, rot, m._PositionsC(None, 2, 0, ok)) == PARAM            # an axis that is not there
    assert _append(m, rot, m._PositionsC(None, 8, 0, ok[:-1] + b"\x08")) == PARAM
    assert _append(m, rot, m._PositionsC(host.BASE + 2, 3, 0, ok)) == ALIGN
    assert _append(m, rot, m._PositionsC(None, 3, 0, ok)) == NULL
    assert _append(m, m._RotaryC(None, 7, 10, 0), m._PositionsC(None, 3, 0, None)) == PARAM


@pytest.mark.parametrize("axes", ["abc", [0, -1], [300], [0.5], 3.5])
def test_axes_that_are_no_numbers(m, axes):
    i = torch.zeros(1, dtype=torch.int32)
    c = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(m.AsvError):
        m.paged_kv_append(c[0, :1], c[0, :1], c, c, i[None], i, torch.zeros(2, dtype=torch.int32), axes=axes)


@pytest.mark.gpu
def test_binding_refuses_positions(m):
    b = Batch([2, 3], [5, 6], heads=(2, 1), dim=32, page=8, seed=2).fill(upto=[5, 6])
    k, v = (x.cuda() for x in b.new_rows())
    rot, at = rotation_table(20, 32).cuda(), torch.zeros(3, 5, dtype=torch.int32, device="cuda")
    axes = [0] * 4 + [1] * 6 + [2] * 6

    def status(**kw):
        args = {**dict(rotary=rot, positions=at, axes=axes), **kw}
        old = b.k_cache.clone()
        with pytest.raises(m.AsvError) as e:
            m.paged_kv_append(k, v, b.k_cache, b.v_cache, b.table, b.cache_len, b.indptr, **args)
        assert torch.equal(old.view(torch.int16), b.k_cache.view(torch.int16))
        return e.value.status

    assert status(rotary=None) == PARAM
    assert status(axes=axes[:-1]) == PARAM
    assert status(axes=axes[:-1] + [3]) == PARAM
    assert status(axes=None) == PARAM                          # which axis a pair takes is not said
    assert status(positions=None) == PARAM
    assert status(positions=at.long()) == DTYPE
    assert status(positions=at[:, :4]) == SHAPE
    assert status(positions=at[None]) == SHAPE
    assert status(positions=at.T.contiguous().T) == SHAPE      # an axis's positions apart
    assert status(positions=at.cpu()) == -1
    assert status(positions=torch.zeros(9, 5, dtype=torch.int32, device="cuda")) == PARAM


# ------------------------------------------------------------------ results

def _check(m, b, axes, pos, *, interleaved=False, with_q=True, views=False, positions=None, limit=None, stream=None):
    """`axes` and `pos` [A, N] on the host; `positions`: the tensor to hand over, if not pos itself."""
    b.fill(upto=b.past)
    before = b.k_cache.cpu(), b.v_cache.cpu()
    k, v = (x.cuda() for x in b.new_rows())
    q = b.q.cuda()
    if views:
        both = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1)
        q, k, v = (x.unflatten(1, (-1, b.dim)) for x in both.split([b.Hq * b.dim, b.Hkv * b.dim, b.Hkv * b.dim], 1))
    half = len(axes)
    table = rotation_table(limit or int(pos.max()) + 1, 2 * half)
    out = m.paged_kv_append(k, v, b.k_cache, b.v_cache, b.table, b.cache_len, b.indptr, q=q if with_q else None,
                            rotary=table.cuda(), interleaved=interleaved,
                            positions=pos.to(torch.int32).cuda() if positions is None else positions, axes=axes,
                            stream=stream)
    torch.cuda.synchronize()
    assert not out.req_status.any()
    pair = torch.arange(half)
    row = pos.long()[torch.tensor(list(axes))].T                          # [N, pairs]
    own = torch.cat([table[row, pair], table[row, half + pair]], 1)       # each token's own row of the table
    kn, vn = b.new_rows()
    want_k, tol_k = rotate64(kn, own, interleaved)
    want_q, tol_q = rotate64(b.q, own, interleaved)
    at = [(b.rows[r][(a + i) // b.page], (a + i) % b.page) for r, (a, n) in enumerate(zip(b.past, b.q_lens))
          for i in range(n)]
    pages, slots = (torch.tensor(x, dtype=torch.long) for x in zip(*at))
    kc, vc = b.k_cache.cpu(), b.v_cache.cpu()
    assert_within(kc[pages, slots], want_k, tol_k, "keys")
    assert torch.equal(vc[pages, slots].view(torch.int16), vn.view(torch.int16))
    if with_q:
        assert_within(out.q, want_q, tol_q, "queries")
    for now, old in zip((kc, vc), before):   # nothing else is touched
        now, old = now.contiguous(), old.contiguous()
        now[pages, slots] = 0
        old[pages, slots] = 0
        assert torch.equal(now.view(torch.int16), old.view(torch.int16))


def _random(b, A, limit, seed=0):
    return torch.randint(0, limit, (A, b.N), generator=torch.Generator().manual_seed(seed))


def _deal(pairs, A, seed):
    return torch.randint(0, A, (pairs,), generator=torch.Generator().manual_seed(seed)).tolist()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("A", [1, 2, 3, 8])
@pytest.mark.parametrize("rot,interleaved", [(64, False), (64, True), (40, False), (10, False), (2, True), (6, True)])
def test_axes_of_the_pairs(m, dtype, A, rot, interleaved):
    b = Batch([3, 1, 0, 18, 40], [5, 0, 9, 16, 31], heads=(6, 2), dim=64, page=16, dtype=dtype, seed=3)
    _check(m, b, _deal(rot // 2, A, rot), _random(b, A, 700, A), interleaved=interleaved)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,heads", [(128, (28, 4)), (128, (32, 8)), (80, (5, 5)), (120, (7, 1)), (8, (1, 1))])
def test_head_layouts(m, dim, heads):
    b = Batch([1, 7, 2], [0, 24, 130], heads=heads, dim=dim, page=24, seed=dim)
    _check(m, b, bytes(_deal(dim // 2, 3, 1)), _random(b, 3, 90), views=True)


@pytest.mark.gpu
def test_a_pair_on_every_table_row(m):
    """The table's first and last rows, and tokens whose slots are far past the table's end."""
    b = Batch([4, 2], [200, 0], heads=(2, 1), dim=32, page=16, seed=1)
    pos = torch.tensor([[0, 9, 9, 0, 1, 9], [9, 0, 9, 0, 9, 9]])
    _check(m, b, [0, 1] * 8, pos, limit=10)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1300, 2500, 5000, 10000])
def test_many_tokens_of_few_heads(m, n):
    """From one to sixteen tokens to a CTA."""
    q_lens = [1, 0, 7, 2, 31, 3, 0, 0, 5, 1]
    q_lens += [n - sum(q_lens) - 40, 37, 3]
    b = Batch(q_lens, [(53 * i) % 90 for i in range(len(q_lens))], heads=(1, 1), dim=16, page=16, seed=n)
    _check(m, b, _deal(4, 3, n), _random(b, 3, 50))


@pytest.mark.gpu
def test_axes_far_apart_rows_behind_and_another_stream(m):
    """Positions as views of a longer buffer, one axis without axes=, keys and values only, a stream of its own."""
    b = Batch([9, 2], [4, 4], heads=(2, 2), dim=32, seed=8)
    pos = _random(b, 3, 60)
    wide = torch.full((5, 40), -5, dtype=torch.int32, device="cuda")
    wide[::2, 3:3 + b.N] = pos.to(torch.int32).cuda()
    torch.cuda.synchronize()
    _check(m, b, [2, 0, 1, 1] * 4, pos, positions=wide[::2, 3:3 + b.N], stream=torch.cuda.Stream())
    b = Batch([9, 2], [4, 4], heads=(2, 2), dim=32, seed=8)
    _check(m, b, [0] * 16, pos[:1], positions=wide[0, 3:3 + b.N], with_q=False)


@pytest.mark.gpu
def test_slots_positions_are_the_default(m):
    """Given the slots' own positions the results are the ordinary call's, bit for bit."""
    b = Batch([3, 1, 0, 18], [5, 0, 9, 16], heads=(6, 2), dim=64, page=16, seed=3).fill(upto=[5, 0, 9, 16])
    k, v = (x.cuda() for x in b.new_rows())
    rot = rotation_table(64, 64).cuda()
    pos = torch.tensor([a + i for a, n in zip(b.past, b.q_lens) for i in range(n)], dtype=torch.int32, device="cuda")
    outs = []
    for kw in ({}, dict(positions=pos), dict(positions=pos[None].repeat(3, 1), axes=[0, 1, 2, 2] * 8)):
        kc, vc = b.k_cache.clone(), b.v_cache.clone()
        out = m.paged_kv_append(k, v, kc, vc, b.table, b.cache_len, b.indptr, q=b.qd, rotary=rot, **kw)
        assert not out.req_status.any()
        outs.append((out.q, kc, vc))
    for got in outs[1:]:
        for x, y in zip(got, outs[0]):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))


@pytest.mark.gpu
def test_a_position_outside_the_table_leaves_its_token_out(m):
    b = Batch([2, 3, 1], [5, 6, 7], heads=(2, 1), dim=32, page=8, seed=2).fill(upto=[5, 6, 7])
    k, v = (x.cuda() for x in b.new_rows())
    pos = torch.zeros(2, 6, dtype=torch.int32, device="cuda")
    pos[0, 3], pos[1, 5] = 10, -1          # request 1's second token, request 2's only one
    b.cache_len[0] = -1                    # (request 0 is left out for its length, whatever its positions)
    pos[:, 0] = 1 << 30
    old, q_out = b.k_cache.clone(), torch.full_like(b.qd, 7.0)
    out = m.PagedAppendOutput(q_out, torch.zeros(3, dtype=torch.int32, device="cuda"))
    m.paged_kv_append(k, v, b.k_cache, b.v_cache, b.table, b.cache_len, b.indptr, q=b.qd, out=out,
                      rotary=rotation_table(10, 32).cuda(), positions=pos, axes=[0, 1] * 8)
    assert out.req_status.tolist() == [m.REQ_BAD_LEN] * 3
    same = (old.view(torch.int16) == b.k_cache.view(torch.int16)).flatten(2).all(-1)
    assert sorted(map(tuple, (~same).nonzero().tolist())) == sorted((b.rows[1][p // 8], p % 8) for p in (6, 8))
    assert [bool((r == 7).all()) for r in q_out] == [True, True, False, True, False, True]
