"""paged_attention against its formula in 64 bits, within the roundings of paged_util.attention64."""
import math

import pytest
import torch

from paged_util import Batch, assert_within, attention64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def asv():
    import speculative_decoding_logit_gb300 as m
    m.build()
    return m


def _run(asv, b, **kw):
    out = asv.paged_attention(b.qd, b.k_cache, b.v_cache, b.table, b.cache_len, b.indptr, **kw)
    torch.cuda.synchronize()
    return out


def _check(asv, b, window=0, scale=None):
    got = _run(asv, b.fill(), window=window, scale=scale)
    assert not got.req_status.any()
    out, lse, tol, ltol = attention64(b, scale, window)
    assert_within(got.out, out, tol, "out")
    assert_within(got.lse, lse, ltol, "lse")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("past", [0, 1, 15, 16, 126, 127, 128, 129, 255, 256, 300, 511])
def test_single_tokens_at_tile_borders(asv, dtype, past):
    _check(asv, Batch([1], [past], heads=(8, 2), dim=128, dtype=dtype, seed=past))


@pytest.mark.parametrize("dim", [8, 24, 40, 64, 72, 80, 96, 120, 128])
@pytest.mark.parametrize("heads", [(1, 1), (7, 1), (6, 3), (16, 2)])
def test_head_layouts(asv, dim, heads):
    _check(asv, Batch([3, 1, 20], [130, 0, 45], heads=heads, dim=dim, page=16, seed=dim))
    _check(asv, Batch([3, 1, 20], [130, 0, 45], heads=heads, dim=dim, page=16, seed=dim, heads_first=True))


@pytest.mark.parametrize("page", [8, 16, 24, 32, 40, 48, 64, 96, 128, 192, 256, 512])
def test_page_sizes(asv, page):
    _check(asv, Batch([5, 2, 33], [290, 7, 111], heads=(4, 2), dim=64, page=page, seed=page))


@pytest.mark.parametrize("q_len", [2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 260])
@pytest.mark.parametrize("group", [1, 4, 5])
def test_chunk_lengths(asv, q_len, group):
    _check(asv, Batch([q_len], [70], heads=(group, 1), dim=64, page=32, seed=q_len))


@pytest.mark.parametrize("window", [1, 2, 17, 100, 128, 129, 1000])
def test_windows(asv, window):
    _check(asv, Batch([1, 4, 90, 0, 150], [400, 129, 3, 60, 0], heads=(4, 2), dim=64, seed=window), window=window)


@pytest.mark.parametrize("seed", range(4))
def test_ragged_batches(asv, seed):
    g = torch.Generator().manual_seed(seed)
    n = 37
    q = torch.randint(0, 6, (n,), generator=g).tolist()
    past = torch.randint(0, 420, (n,), generator=g).tolist()
    q[0], q[5], q[-1] = 0, 140, 0
    _check(asv, Batch(q, past, heads=(8, 2), dim=128, page=[16, 48, 64, 8][seed], seed=seed,
                      dtype=[torch.bfloat16, torch.float16][seed % 2]))


@pytest.mark.parametrize("group,q_lens,past", [
    (32, [1, 1], [257, 0]), (10, [3, 3, 3], [130, 1200, 61]), (10, [6, 0, 3, 3], [130, 5, 0, 1000]), (1, [40, 24], [0, 300]),
    (5, [7, 5, 6], [96, 129, 31]), (31, [1] * 5, [0, 31, 32, 33, 640]), (12, [2, 2], [2000, 127]), (3, [10], [4000]),
])
@pytest.mark.parametrize("window", [0, 70])
def test_few_rows(asv, group, q_lens, past, window):
    """At most 32 rows to an item on average: the warps divide a tile's positions among them."""
    for dim, dtype in ((128, torch.bfloat16), (64, torch.float16), (40, torch.bfloat16)):
        _check(asv, Batch(q_lens, past, heads=(2 * group, 2), dim=dim, page=24, dtype=dtype, seed=group), window=window)


def test_long_split_context(asv):
    """Few rows over many keys: the work of one request is split and joined."""
    _check(asv, Batch([2], [9000], heads=(2, 1), dim=128, page=64, seed=1))
    _check(asv, Batch([1, 1], [7001, 40], heads=(1, 1), dim=64, page=16, seed=2))


def test_long_prompt(asv):
    _check(asv, Batch([700, 300], [0, 17], heads=(3, 1), dim=64, page=64, seed=5))


def test_many_heads_to_one(asv):
    _check(asv, Batch([1, 3], [200, 10], heads=(128, 1), dim=64, seed=5))
    _check(asv, Batch([2, 5], [200, 10], heads=(100, 1), dim=64, seed=6))


@pytest.mark.parametrize("gain,scale", [(6.0, None), (1.0, 1.0), (0.01, None)])
def test_peaked_and_flat_scores(asv, gain, scale):
    """Scores far apart (the running maximum moves by hundreds), and all alike."""
    _check(asv, Batch([4, 40], [500, 260], heads=(4, 2), dim=64, gain=gain, seed=9), scale=scale)


@pytest.mark.parametrize("heads", [(4, 2), (20, 2), (64, 2)])
def test_rising_scores_move_the_maximum_in_every_tile(asv, heads):
    b = Batch([3], [1200], heads=heads, dim=64, seed=11)
    ramp = torch.linspace(0, 8, 1203)[:, None, None]
    b.q = b.q.abs().clamp(min=0.25)
    b.k[0] = (b.k[0].abs().float() * ramp).to(b.dtype)
    _check(asv, b, scale=0.25)


def test_infinite_scores_weigh_nothing(asv):
    """A key of -inf products has weight 0; the formula holds over the rest."""
    b = Batch([2], [200], heads=(2, 1), dim=64, seed=12)
    b.q = b.q.abs() + 0.5
    for j in (0, 64, 130):
        b.k[0][j, 0, 0] = -math.inf
    got = _run(asv, b.fill())
    keep = torch.ones(202, dtype=torch.bool)
    keep[[0, 64, 130]] = False
    for i in range(2):
        kk, vv = b.k[0][:201 + i, 0][keep[:201 + i]].double(), b.v[0][:201 + i, 0][keep[:201 + i]].double()
        p = torch.softmax(b.q[i].double() @ kk.T * 64 ** -0.5, -1)
        want = p @ vv
        tol = 2.0 ** -8 * (want.abs() + p @ vv.abs()) * 1.05
        assert_within(got.out[i], want, tol, "out")


def test_nan_where_no_token_looks(asv):
    """NaN and infinities at positions after a token (later tokens of its own chunk), before its window,
    and in pages the window has left (their table entries out of range) leave it alone."""
    b = Batch([40, 3], [150, 700], heads=(4, 2), dim=64, seed=13)
    w = 90
    b.fill()
    want = attention64(b, None, w)
    for b2, at, rows in ((0, 175, range(0, 25)), (1, 701, range(40, 41))):
        for bad in (math.nan, math.inf, -math.inf):
            k, v = b.k_cache.clone(), b.v_cache.clone()
            n = b.past[b2] + b.q_lens[b2]
            for j in range(at, n):
                k[b.rows[b2][j // 16], j % 16] = bad
                v[b.rows[b2][j // 16], j % 16] = bad
            for j in range(0, max(0, b.past[b2] + 1 - w)):
                k[b.rows[b2][j // 16], j % 16] = bad
                v[b.rows[b2][j // 16], j % 16] = bad
            table = b.table.clone()
            table[b2, :max(0, b.past[b2] + 1 - w) // 16] = -1
            got = asv.paged_attention(b.qd, k, v, table, b.cache_len, b.indptr, window=w)
            assert not got.req_status.any()
            rows = list(rows)
            assert_within(got.out[rows], want[0][rows], want[2][rows], "out")
            assert_within(got.lse[rows], want[1][rows], want[3][rows], "lse")
            other = [r for r in range(43) if (r < 40) != (b2 == 0)]
            assert_within(got.out[other], want[0][other], want[2][other], "the other request")


@pytest.mark.parametrize("heads,q_lens", [((4, 1), [300, 20, 150]), ((2, 2), [260, 257, 5, 390]), ((4, 1), [6, 6, 3, 9]),
                                          ((30, 2), [2, 2])])
def test_nan_in_later_tokens_of_long_chunks(asv, heads, q_lens):
    """The last third of every chunk holds NaN keys and values: the tokens before it are left alone, whichever
    row tiles and items they share with it, and every one from there on is NaN."""
    b = Batch(q_lens, [70, 0, 200, 11][:len(q_lens)], heads=heads, dim=64, page=32, seed=21).fill()
    want = attention64(b)
    clean, bad = [], []
    for r, (a, n) in enumerate(zip(b.past, b.q_lens)):
        cut = n - n // 3
        for j in range(a + cut, a + n):
            for c in (b.k_cache, b.v_cache):
                c[b.rows[r][j // 32], j % 32] = math.nan
        clean += range(b.starts[r], b.starts[r] + cut)
        bad += range(b.starts[r] + cut, b.starts[r] + n)
    got = _run(asv, b)
    assert not got.req_status.any()
    assert_within(got.out[clean], want[0][clean], want[2][clean], "out")
    assert_within(got.lse[clean], want[1][clean], want[3][clean], "lse")
    assert bool(got.out[bad].isnan().all())


def test_infinite_values_stay_with_their_rows_and_columns(asv):
    """Infinities of both signs among the values of a chunk's own tokens: a row that sees one of a column is
    infinite there, NaN where it sees both signs, and the others are left alone."""
    b = Batch([90], [140], heads=(2, 1), dim=64, seed=22)
    b.v[0][150, 0, 3] = math.inf
    b.v[0][171, 0, 3] = -math.inf
    b.v[0][171, 0, 9] = -math.inf
    b.fill()
    keep = b.v[0].clone()
    b.v[0] = torch.where(keep.isinf(), 0, keep)
    want = attention64(b)
    got = _run(asv, b)
    pos = torch.arange(140, 230)[:, None]
    col = torch.arange(64)[None]
    plus, minus = (col == 3) & (pos >= 150), ((col == 3) | (col == 9)) & (pos >= 171)
    out = got.out.float().cpu()
    for h in range(2):
        o = out[:, h]
        assert torch.equal(o.isnan(), plus & minus)
        assert torch.equal(o == math.inf, plus & ~minus) and torch.equal(o == -math.inf, minus & ~plus)
        ok = ~(plus | minus)
        assert bool(((o.double() - want[0][:, h]).abs() <= want[2][:, h])[ok].all())


def test_nan_among_the_keys_reaches_its_rows(asv):
    b = Batch([4], [100], heads=(2, 2), dim=64, seed=14).fill()
    b.v_cache[b.rows[0][102 // 16], 102 % 16, 1, 5] = math.nan
    b.k_cache[b.rows[0][103 // 16], 103 % 16, 0, 2] = math.nan
    got = _run(asv, b)
    nan = got.out.isnan()
    want = torch.zeros_like(nan)
    want[2:, 1, 5] = True
    want[3, 0, :] = True
    assert torch.equal(nan, want)


def test_strided_queries_and_outputs_and_no_lse(asv):
    b = Batch([3, 30], [77, 5], heads=(4, 2), dim=64, seed=15).fill()
    ref = _run(asv, b)
    wide = torch.zeros(b.N, 3, b.Hq, 64 + 8, dtype=b.dtype, device="cuda")
    wide[:, 1, :, :64] = b.qd
    room = torch.full((b.N, b.Hq, 2, 64), 7.0, dtype=b.dtype, device="cuda")
    out = asv.PagedAttentionOutput(room[:, :, 1], None, torch.zeros(2, dtype=torch.int32, device="cuda"))
    asv.paged_attention(wide[:, 1, :, :64], b.k_cache, b.v_cache, b.table, b.cache_len, b.indptr, out=out)
    assert torch.equal(out.out, ref.out)
    assert bool((room[:, :, 0] == 7.0).all())


def test_bad_lengths_and_pages_are_flagged(asv):
    b = Batch([2, 3, 2, 4, 1], [50, 60, 70, 80, 200], heads=(2, 1), dim=64, page=8, seed=2).fill()
    good = _run(asv, b)
    b.cache_len[1] = -1
    b.table[2, 3] = -7
    b.cache_len[3] = b.table.shape[1] * 8 - 3
    got = _run(asv, b)
    assert got.req_status.tolist() == [0, asv.REQ_BAD_LEN, asv.REQ_BAD_PAGE, asv.REQ_BAD_LEN, 0]
    for r in (0, 1, 11):   # requests 0 and 4
        assert torch.equal(got.out[r], good.out[r]) and torch.equal(got.lse[r], good.lse[r])
    for r in (2, 3, 4, 7, 8, 9, 10):
        assert not got.out[r].any() and bool((got.lse[r] == -math.inf).all())


def test_broken_indptr_is_flagged(asv):
    b = Batch([2, 3, 4], [50, 60, 70], heads=(2, 1), dim=64, page=8, seed=2).fill()
    for rows, want in (([0, 2, 1, 9], [0, 1, 0]), ([0, 2, 5, 99], [0, 0, 1]), ([-4, 2, 5, 9], [1, 0, 0])):
        ptr = torch.tensor(rows, dtype=torch.int32, device="cuda")
        out = asv.paged_attention(b.qd, b.k_cache, b.v_cache, b.table, b.cache_len, ptr)
        torch.cuda.synchronize()
        assert [int(x != 0) for x in out.req_status.tolist()] == want


def test_the_same_call_gives_the_same_bits(asv):
    b = Batch([1, 9, 300, 2], [3000, 500, 90, 1200], heads=(8, 2), dim=128, page=16, seed=16).fill()
    ref = _run(asv, b)
    for _ in range(5):
        got = _run(asv, b)
        assert torch.equal(got.out, ref.out) and torch.equal(got.lse, ref.lse)


def test_other_stream_and_own_workspace(asv):
    b = Batch([1, 9], [2000, 500], heads=(8, 2), dim=128, page=16, seed=17).fill()
    ref = _run(asv, b)
    s = torch.cuda.Stream()
    ws = torch.zeros(asv.paged_workspace_bytes(8, 2, 128), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        got = asv.paged_attention(b.qd, b.k_cache, b.v_cache, b.table, b.cache_len, b.indptr, stream=s, workspace=ws)
    s.synchronize()
    assert torch.equal(got.out, ref.out) and torch.equal(got.lse, ref.lse)


def test_offsets_past_32_bits(asv):
    """Pages whose element offsets pass 2^32."""
    page, H, D = 64, 8, 128
    n_pages = (1 << 32) // (page * H * D) + 40
    k, v = (torch.empty(n_pages, page, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    b = Batch([2], [300], heads=(8, 8), dim=D, page=page, seed=18)
    rows = list(range(n_pages - len(b.rows[0]), n_pages))
    b.fill()
    for j, r in enumerate(rows):
        k[r], v[r] = b.k_cache[b.rows[0][j]], b.v_cache[b.rows[0][j]]
    b.k_cache, b.v_cache = k, v
    b.table = torch.tensor([rows], dtype=torch.int32, device="cuda")
    got = _run(asv, b)
    out, lse, tol, ltol = attention64(b)
    assert_within(got.out, out, tol, "out")
    assert_within(got.lse, lse, ltol, "lse")


def test_append_then_attend_in_a_replayed_graph(asv):
    """A decoding step (append, attend, advance) captured once and replayed: the lengths live on the
    device, so every replay works on the cache the one before left."""
    from paged_util import rotation_table
    steps, K1 = 3, 3
    b = Batch([K1 * steps] * 2, [21, 140], heads=(4, 2), dim=64, seed=19)
    b.fill(upto=b.past)
    table = rotation_table(200, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    indptr = torch.tensor([0, K1, 2 * K1], **i32)
    kn, vn = b.new_rows()
    pick = [[r * K1 * steps + s * K1 + i for r in range(2) for i in range(K1)] for s in range(steps)]
    q, k, v = (torch.empty(2 * K1, h, 64, dtype=b.dtype, device="cuda") for h in (4, 2, 2))
    length = b.cache_len.clone()
    rot = table.cuda()
    app = asv.PagedAppendOutput(torch.empty_like(q), torch.zeros(2, **i32))
    att = asv.PagedAttentionOutput(torch.empty_like(q), torch.empty(2 * K1, 4, device="cuda"), torch.zeros(2, **i32))
    ws = torch.zeros(asv.paged_workspace_bytes(4, 2, 64), dtype=torch.uint8, device="cuda")

    def step():
        asv.paged_kv_append(k, v, b.k_cache, b.v_cache, b.table, length, indptr, q=q, rotary=rot, out=app)
        asv.paged_attention(app.q, b.k_cache, b.v_cache, b.table, length, indptr, out=att, workspace=ws)
        length.add_(K1)

    def load(s):
        for dst, src in ((q, b.q), (k, kn), (v, vn)):
            dst.copy_(src[pick[s]])

    s0 = torch.cuda.Stream()
    s0.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s0):
        load(0)
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    length.copy_(b.cache_len)
    outs = []
    for s in range(steps):
        load(s)
        g.replay()
        outs.append((att.out.clone(), att.lse.clone(), app.q.clone()))
    torch.cuda.synchronize()
    assert not app.req_status.any() and not att.req_status.any()
    # the formula over what the cache and the rotated queries hold
    for r in range(2):
        for p in range(b.past[r], b.past[r] + K1 * steps):
            b.k[r][p] = b.k_cache[b.rows[r][p // 16], p % 16].cpu()
    for s in range(steps):
        b.q[pick[s]] = outs[s][2].cpu()
    out, lse, tol, ltol = attention64(b)
    for s in range(steps):
        assert_within(outs[s][0], out[pick[s]], tol[pick[s]], "out")
        assert_within(outs[s][1], lse[pick[s]], ltol[pick[s]], "lse")
