"""paged_kv_append against the same writes made one by one, rotations in 64 bits: the appended slots and
the queries within the roundings of paged_util.rotate64, values and every other slot bit for bit."""
import pytest
import torch

from paged_util import Batch, assert_within, rotate64, rotation_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def asv():
    import speculative_decoding_logit_gb300 as m
    m.build()
    return m


def _bits(x):
    return x.contiguous().view(torch.int16).cpu()


def _check(asv, b, *, rot=None, interleaved=False, with_q=True, views=False, stream=None):
    b.fill(upto=b.past)
    before = b.k_cache.cpu(), b.v_cache.cpu()
    k, v = (x.cuda() for x in b.new_rows())
    q = b.q.cuda()
    if views:  # q, k, v as views of one projection's output, heads apart
        both = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1)
        q, k, v = (x.unflatten(1, (-1, b.dim)) for x in both.split([b.Hq * b.dim, b.Hkv * b.dim, b.Hkv * b.dim], 1))
    table = None if rot is None else rotation_table(max(a + n for a, n in zip(b.past, b.q_lens)), rot)
    out = asv.paged_kv_append(k, v, b.k_cache, b.v_cache, b.table, b.cache_len, b.indptr, q=q if with_q else None,
                              rotary=None if rot is None else table.cuda(), interleaved=interleaved, stream=stream)
    torch.cuda.synchronize()
    assert not out.req_status.any()
    pos = torch.tensor([a + i for a, n in zip(b.past, b.q_lens) for i in range(n)], dtype=torch.long)
    kn, vn = b.new_rows()
    if rot is None:
        want_k, tol_k, want_q, tol_q = kn.double(), kn.double() * 0, b.q.double(), b.q.double() * 0
    else:
        want_k, tol_k = rotate64(kn, table[pos], interleaved)
        want_q, tol_q = rotate64(b.q, table[pos], interleaved)
    at = [(b.rows[r][(a + i) // b.page], (a + i) % b.page) for r, (a, n) in enumerate(zip(b.past, b.q_lens))
          for i in range(n)]
    pages, slots = (torch.tensor(x, dtype=torch.long) for x in zip(*at))
    kc, vc = b.k_cache.cpu(), b.v_cache.cpu()
    assert_within(kc[pages, slots], want_k, tol_k, "keys")
    assert torch.equal(_bits(vc[pages, slots]), _bits(vn))
    if with_q:
        assert_within(out.q, want_q, tol_q, "queries")
    else:
        assert out.q is None
    for now, old in zip((kc, vc), before):   # nothing else is touched
        now, old = now.contiguous(), old.contiguous()
        now[pages, slots] = 0
        old[pages, slots] = 0
        assert torch.equal(_bits(now), _bits(old))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rot,interleaved", [(None, False), (64, False), (64, True), (32, False), (16, True),
                                             (10, False), (6, True), (30, False), (2, False), (24, False), (56, False), (8, False)])
def test_rotations(asv, dtype, rot, interleaved):
    b = Batch([3, 1, 0, 18, 40], [5, 0, 9, 16, 31], heads=(6, 2), dim=64, page=16, dtype=dtype, seed=3)
    _check(asv, b, rot=rot, interleaved=interleaved)


@pytest.mark.parametrize("dim", [8, 40, 64, 80, 120, 128])
@pytest.mark.parametrize("heads", [(1, 1), (5, 5), (28, 4), (64, 8)])
def test_head_layouts(asv, dim, heads):
    b = Batch([1, 7, 2], [0, 24, 130], heads=heads, dim=dim, page=24, seed=dim)
    _check(asv, b, rot=dim, views=True)
    b = Batch([1, 7, 2], [0, 24, 130], heads=heads, dim=dim, page=24, heads_first=True, seed=dim)
    _check(asv, b, rot=max(2, dim // 4 // 2 * 2), interleaved=True)


@pytest.mark.parametrize("n", [1300, 2500, 5000, 10000])
def test_many_tokens_of_few_heads(asv, n):
    """From one to sixteen tokens to a CTA, which take in one request's end and several others."""
    q_lens = [1, 0, 7, 2, 31, 3, 0, 0, 5, 1]
    q_lens += [n - sum(q_lens) - 40, 37, 3]
    b = Batch(q_lens, [(53 * i) % 90 for i in range(len(q_lens))], heads=(1, 1), dim=16, page=16, seed=n)
    _check(asv, b, rot=8)


@pytest.mark.parametrize("page", [8, 16, 48, 128, 256])
def test_pages_and_single_tokens(asv, page):
    b = Batch([1] * 300, [(37 * i) % 300 for i in range(300)], heads=(2, 1), dim=16, page=page, seed=page)
    _check(asv, b, rot=16)


def test_keys_and_values_only_on_another_stream(asv):
    b = Batch([9, 2], [4, 4], heads=(2, 2), dim=32, seed=8)
    s = torch.cuda.Stream()
    _check(asv, b, rot=32, with_q=False, stream=s)


def test_long_chunk(asv):
    b = Batch([1500, 1, 700], [3, 50, 0], heads=(3, 1), dim=64, page=64, seed=4)
    _check(asv, b, rot=64, views=True)


def test_bad_lengths_and_pages_are_flagged_and_left_out(asv):
    b = Batch([2, 3, 2, 4, 1], [5, 6, 7, 8, 20], heads=(2, 1), dim=32, page=8, seed=2)
    b.fill(upto=b.past)
    k, v = (x.cuda() for x in b.new_rows())
    table = rotation_table(20, 32).cuda()         # request 4's position 20 is past its last row
    b.cache_len[1] = -1                           # request 1: a negative length
    b.table[2, 0] = -7                            # request 2: bad pages where its tokens go
    b.table[2, 1] = b.k_cache.shape[0]
    b.cache_len[3] = b.table.shape[1] * 8 - 3     # request 3: past the block table
    old = b.k_cache.clone()
    out = asv.paged_kv_append(k, v, b.k_cache, b.v_cache, b.table, b.cache_len, b.indptr, q=b.qd, rotary=table)
    assert out.req_status.tolist() == [0, asv.REQ_BAD_LEN, asv.REQ_BAD_PAGE, asv.REQ_BAD_LEN, asv.REQ_BAD_LEN]
    same = (_bits(old) == _bits(b.k_cache)).flatten(2).all(-1)
    changed = (~same).nonzero().tolist()
    assert sorted(map(tuple, changed)) == sorted((b.rows[0][p // 8], p % 8) for p in (5, 6))


def test_broken_indptr_is_flagged(asv):
    b = Batch([2, 3, 4], [5, 6, 7], heads=(2, 1), dim=32, page=8, seed=2).fill(upto=[5, 6, 7])
    k, v = (x.cuda() for x in b.new_rows())
    for rows, want in (([0, 2, 1, 9], [0, 1, 0]), ([0, 2, 5, 99], [0, 0, 1]), ([-4, 2, 5, 9], [1, 0, 0])):
        ptr = torch.tensor(rows, dtype=torch.int32, device="cuda")
        out = asv.paged_kv_append(k, v, b.k_cache, b.v_cache, b.table, b.cache_len, ptr)
        assert [int(x != 0) for x in out.req_status.tolist()] == want
