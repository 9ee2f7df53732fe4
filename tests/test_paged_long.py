"""paged_attention with long pieces: a CTA's run holds many key tiles, the ring of tiles goes round, references move within a
piece, and runs are cut evenly.  Every case states, by the split worked out here, that it is what it is meant to be."""
import math

import pytest
import torch

import test_paged_checked as small
from paged_long import TILE, LongBatch, Plan, assert_requests, attention64_wide

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def asv():
    import speculative_decoding_logit_gb300 as m
    m.build()
    return m


def _spread(n, lo, hi):
    """n lengths from lo to hi, evenly by their logarithm, in a scattered order."""
    return [int(lo * (hi / lo) ** (((i * 37) % n) / max(n - 1, 1))) for i in range(n)]


# q_lens, past, heads, dim, page, type, window: two row tiles, one, divided
TWO = [
    ([1500, 700], [5000, 3000], (8, 2), 64, 16, BF, 0),
    ([1000, 650, 40, 0, 1111], [2500, 4100, 3000, 70, 900], (16, 2), 128, 24, FP, 0),
    ([1200, 900, 575], [6000, 777, 5600], (10, 2), 80, 64, BF, 0),
    ([1900, 1700, 1800], [3000, 2500, 1], (8, 4), 128, 128, BF, 1500),
]
ONE = [
    ([5, 7, 9, 11, 3, 8] * 5, _spread(30, 2500, 9500), (16, 2), 128, 16, BF, 0),
    ([11] * 24, _spread(24, 3000, 12000), (16, 2), 64, 32, FP, 0),
    ([1] * 63 + [500], _spread(64, 1000, 6000), (16, 4), 128, 64, BF, 0),
    ([13, 17, 20, 0] * 16, _spread(64, 3000, 9000), (12, 4), 96, 48, FP, 1777),
]
DIVIDED = [
    ([1] * 140, _spread(140, 1, 12000), (8, 2), 128, 16, BF, 0),
    ([3] * 40, _spread(40, 2500, 9000), (16, 2), 64, 24, FP, 0),
    ([2, 3, 1, 2] * 2, _spread(8, 30000, 60000), (10, 1), 128, 64, BF, 0),
    ([2] * 100, _spread(100, 900, 9000), (12, 4), 40, 40, FP, 1300),
]
CASES = [(k, i) for k, cases in (("two", TWO), ("one", ONE), ("divided", DIVIDED)) for i in range(len(cases))]


def _case(kind, i, gain=1.0):
    q, past, heads, dim, page, dtype, window = {"two": TWO, "one": ONE, "divided": DIVIDED}[kind][i]
    b = LongBatch(q, past, heads=heads, dim=dim, page=page, dtype=dtype, seed=i, gain=gain)
    plan = Plan(b, window)
    assert (plan.two, plan.divided) == (kind == "two", kind == "divided")
    assert plan.run > 16 and plan.units % len(plan.pieces) != 0
    whole, cut = plan.longest()
    assert cut >= 3 and max(whole, cut) >= 10
    return b, plan, window


@pytest.mark.parametrize("kind,i", CASES)
def test_long_pieces(asv, kind, i):
    b, plan, window = _case(kind, i)
    b.fill()
    ws = torch.zeros(asv.paged_workspace_bytes(b.Hq, b.Hkv, b.dim), dtype=torch.uint8, device="cuda")
    got = asv.paged_attention(*b.args(), window=window, workspace=ws)
    assert not got.req_status.any()
    assert_requests(b, got, attention64_wide(b, window=window))
    assert not ws[:4096].any()   # tickets
    again = asv.paged_attention(*b.args(), window=window, workspace=ws)
    assert torch.equal(got.out, again.out) and torch.equal(got.lse, again.lse)
    assert not ws[:4096].any()


@pytest.mark.parametrize("kind,i", [("two", 0), ("two", 3), ("one", 0), ("one", 3), ("divided", 0), ("divided", 1), ("divided", 3)])
def test_rising_scores_move_the_reference_within_a_piece(asv, kind, i):
    b, plan, window = _case(kind, i)
    b.qd = b.qd.abs().clamp(min=0.5)
    for r in range(b.B):
        n = b.k[r].shape[0]
        ramp = torch.linspace(0, n / TILE * 0.4, n, device="cuda")[:, None, None]
        b.k[r] = (b.k[r].abs().float() * ramp).to(b.dtype)
    scale = 16.0 / b.dim
    # the longest piece's first row: how often a tile's maximum passes the reference by more than 8 (in log2)
    r, h, t, _, t0, t1, _ = max(plan.all(), key=lambda p: p[5] - p[4])
    row = b.starts[r] + t
    s = (b.k[r][:b.past[r] + t + 1, h].double() @ b.qd[row, h * b.group].double()) * scale / math.log(2)
    lo = max(0, b.past[r] + t - window + 1) if window else 0
    ref, moves, kept = -math.inf, 0, 0
    for x in range(t0, t1):
        tile = s[max(x * TILE, lo):(x + 1) * TILE]
        if len(tile) and float(tile.max()) > ref + 8:
            ref, moves = float(tile.max()), moves + 1
        else:
            kept += 1
    assert moves >= 4
    b.fill()
    got = asv.paged_attention(*b.args(), window=window, scale=scale)
    assert not got.req_status.any()
    assert_requests(b, got, attention64_wide(b, scale=scale, window=window))


@pytest.mark.parametrize("kind,i", [("two", 1), ("two", 3), ("one", 2), ("one", 3), ("divided", 0), ("divided", 3)])
def test_values_that_are_not_finite_within_long_pieces(asv, kind, i):
    """Infinities and NaN in the first, the middle and the last tile of long pieces, at the window's edge and among the
    chunk's own tokens: a row's column is infinite or NaN where the row attends to them and right everywhere else."""
    b, plan, window = _case(kind, i, gain=0.5)
    finite = [v.clone() for v in b.v]
    long_ones = sorted(plan.all(), key=lambda p: p[4] - p[5])[:4]
    touched = set()
    for j, (r, h, t, count, t0, t1, _) in enumerate(long_ones):
        assert t1 - t0 >= 3
        touched.add(r)
        pos0, last = b.past[r] + t, b.past[r] + t + count - 1
        lo = max(0, pos0 - window + 1) if window else 0
        at = [t0 * TILE + 5, (t0 + t1) // 2 * TILE + 77, (t1 - 1) * TILE + 9, pos0, last, lo, lo + count // 2]
        for n, p in enumerate(at):
            p = min(max(p, lo), last)
            b.v[r][p, h, (3 * n + j) % b.dim] = [math.inf, -math.inf, math.nan][(n + j) % 3]
            b.v[r][p, h, 30] = math.inf if n % 2 else -math.inf
    b.fill()
    got = asv.paged_attention(*b.args(), window=window)
    assert not got.req_status.any()
    odd = b.v
    b.v = finite
    want = attention64_wide(b, window=window)
    for r, (o, lse, tol, ltol) in want.items():
        rows = slice(b.starts[r], b.starts[r + 1])
        out = got.out[rows].double()
        assert bool(((got.lse[rows].double() - lse).abs() <= ltol).all())
        pos = b.past[r] + torch.arange(b.q_lens[r], device="cuda")[:, None]
        key = torch.arange(b.past[r] + b.q_lens[r], device="cuda")[None]
        seen = (key <= pos) & ((key > pos - window) if window else True)
        hit = lambda x: (torch.einsum("nk,khd->nhd", seen.double(), x.double()) > 0).repeat_interleave(b.group, 1)
        plus, minus, nan = hit(odd[r] == math.inf), hit(odd[r] == -math.inf), hit(odd[r].isnan())
        nan |= plus & minus
        assert bool((plus | minus | nan).any()) == (r in touched)
        assert torch.equal(out.isnan(), nan)
        assert torch.equal(out == math.inf, plus & ~nan) and torch.equal(out == -math.inf, minus & ~nan)
        ok = ~(plus | minus | nan)
        assert bool(((out - o).abs() <= tol)[ok].all())


libs = small.libs


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("q_lens,past,heads,dim,page,window", [
    ([1300, 1100], [4500, 3000], (8, 2), 64, 16, 0),
    ([1] * 50, [70 * ((i * 37) % 50) + 200 for i in range(50)], (8, 4), 128, 24, 0),
    ([6] * 50, [2500 + 40 * i for i in range(50)], (20, 2), 64, 64, 2900),
])
def test_no_index_of_long_pieces_leaves_its_buffer(libs, dtype, q_lens, past, heads, dim, page, window):
    b = type("Shape", (), dict(q_lens=q_lens, past=past, N=sum(q_lens), B=len(q_lens), group=heads[0] // heads[1], Hkv=heads[1]))
    assert Plan(b, window).run > 16
    small.test_no_index_leaves_its_buffer(libs, dtype, q_lens, past, heads, dim, page, window, False)
