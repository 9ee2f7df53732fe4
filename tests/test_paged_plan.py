"""paged_plan against the same steps taken one by one in Python (whole numbers: equal), its refusals, and what it leaves alone."""
import ctypes as C
import random

import pytest
import torch

import test_paged_refusals as host

NULL, SHAPE, ALIGN, DTYPE, PARAM = 1, 2, 3, 4, 5
m = host.m


# ------------------------------------------------------------------ refusals, on the host

def _pool(m, **kw):
    p = dict(block_table=None, max_pages=4, block_table_stride=4, page_size=16, held=None, free_pages=None, pool_size=8,
             free_count=None)
    p.update(kw)
    return m._PagePoolC(**p)


def _plan(m, pool=None, B=2, N=3, **kw):
    names = ("release", "indptr", "slots", "positions", "requests", "status")
    a = {**dict.fromkeys(("cache_len", "new_len") + names), **kw}
    pool = pool or _pool(m)
    return m.library().paged_plan(a["cache_len"], a["new_len"], B, C.addressof(pool), a["release"], N, a["indptr"],
                                  a["slots"], a["positions"], a["requests"], a["status"], None)


def test_sizes(m):
    for kw in (dict(B=-1), dict(B=16385), dict(N=-1), dict(N=(1 << 30) + 1)):
        assert _plan(m, **kw) == SHAPE
    for kw in (dict(max_pages=-1), dict(pool_size=-1), dict(page_size=0), dict(max_pages=1 << 28),
               dict(block_table_stride=3), dict(block_table_stride=-4)):
        assert _plan(m, _pool(m, **kw)) == SHAPE
    assert _plan(m, _pool(m, block_table_stride=0), B=1) == NULL  # a single row's stride is not looked at
    assert _plan(m, B=0) == 0
    assert _plan(m) == NULL
    assert m.library().paged_plan(None, None, 1, None, None, 0, None, None, None, None, None, None) == NULL


def test_alignment(m):
    odd = host.BASE + 2
    for name in ("cache_len", "new_len", "indptr", "positions", "requests", "status"):
        assert _plan(m, **{name: odd}) == ALIGN
    assert _plan(m, slots=host.BASE + 4) == ALIGN
    for name in ("block_table", "held", "free_pages", "free_count"):
        assert _plan(m, _pool(m, **{name: odd})) == ALIGN


def test_binding_refuses_host_tensors_and_missing_rows(m):
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(m.AsvError):
        m.paged_plan(i, i, i[None], i, i, i, 16, max_tokens=3)


@pytest.mark.gpu
def test_binding_refuses_shapes_and_types(m):
    s = State([3, 4], [1, 2], 16, width=3)
    before = s.tensors()

    def status(**kw):
        a = dict(cache_len=s.cache_len, new_len=s.new_len, block_table=s.table, held=s.held, free_pages=s.free,
                 free_count=s.count, page_size=16, max_tokens=5)
        a.update(kw)
        with pytest.raises(m.AsvError) as e:
            m.paged_plan(**a)
        return e.value.status

    assert status(cache_len=s.cache_len[:1]) == SHAPE
    assert status(new_len=s.new_len.long()) == DTYPE
    assert status(held=s.held[:, None]) == SHAPE
    assert status(free_count=torch.zeros(2, dtype=torch.int32, device="cuda")) == SHAPE
    assert status(free_pages=s.free.long()) == DTYPE
    assert status(free_pages=s.free[None]) == SHAPE
    assert status(block_table=s.table.T.contiguous().T) == SHAPE
    assert status(block_table=s.table[0]) == SHAPE
    assert status(release=torch.zeros(2, dtype=torch.int32, device="cuda")) == DTYPE
    assert status(release=torch.zeros(2, dtype=torch.bool)) == -1
    assert status(max_tokens=None) == PARAM
    assert status(max_tokens=-1) == SHAPE
    assert status(page_size=0) == SHAPE
    assert status(page_size=None) == PARAM
    out = m.PagedPlanOutput(torch.zeros(3, dtype=torch.int32, device="cuda"), None, None, None,
                            torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert status(out=out, max_tokens=None) == PARAM
    out.slots = torch.zeros(5, dtype=torch.int32, device="cuda")
    assert status(out=out, max_tokens=None) == DTYPE
    out.slots, out.indptr = None, out.indptr[:2]
    assert status(out=out) == SHAPE
    assert all(torch.equal(x, y) for x, y in zip(s.tensors(), before))


# ------------------------------------------------------------------ results

class State:
    """Requests with `past` cached tokens on random pages (`extra[b]` pages held beyond them), a pool of the rest."""

    def __init__(self, past, new, page, *, width=None, spare=40, extra=None, released=None, seed=0, stride=0):
        B = len(past)
        released = released or [0] * B                  # pages that the place's former request held; 0: not released
        self.page = page
        held = [r if r else -(-p // page) + (extra[b] if extra else 0) for b, (p, r) in enumerate(zip(past, released))]
        need = [-(-(p + max(n, 0)) // page) for p, n in zip(past, new)]
        width = width or max(need + held + [1])
        total = sum(held) + spare
        order = list(range(total))
        random.Random(seed).shuffle(order)
        rows, at = [], 0
        for h in held:
            rows.append(order[at:at + h] + [-9] * (width - h))
            at += h
        i32 = dict(dtype=torch.int32, device="cuda")
        whole = torch.full((B, width + stride), -77, **i32)
        self.table = whole[:, :width]
        self.whole = whole
        self.table.copy_(torch.tensor(rows, **i32).reshape(B, width))
        self.held, self.cache_len, self.new_len = (torch.tensor(x, **i32) for x in (held, past, new))
        self.free = torch.tensor(order[at:] + [-5] * at, **i32)
        self.count = torch.tensor([total - at], **i32)
        self.release = torch.tensor([r > 0 for r in released], device="cuda") if any(released) else None

    def tensors(self):
        return [x.clone() for x in (self.whole, self.held, self.free, self.count, self.cache_len, self.new_len)]

    def expected(self, N, m):
        table, held, free, top = self.table.tolist(), self.held.tolist(), self.free.tolist(), int(self.count)
        past, new = self.cache_len.tolist(), self.new_len.tolist()
        B, width = self.table.shape
        over = self.release.tolist() if self.release is not None else [False] * B
        status = [0] * B
        for b in range(B):
            if over[b] and 0 <= held[b] <= width:
                for j in range(held[b]):
                    free[top], table[b][j] = table[b][j], -1
                    top += 1
                held[b] = 0
        room, asked, rows = top, 0, 0
        slots, positions, requests, indptr = [], [], [], [0]
        for b in range(B):
            ok = 0 <= held[b] <= width and 0 <= past[b] <= held[b] * self.page and new[b] >= 0 and \
                past[b] + new[b] <= width * self.page
            if not ok:
                status[b] = m.REQ_BAD_LEN
            else:
                need = max(0, -(-(past[b] + new[b]) // self.page) - held[b])
                asked, rows = asked + need, rows + new[b]
                if (need == 0 or asked <= room) and rows <= N:
                    for _ in range(need):
                        top -= 1
                        table[b][held[b]] = free[top]
                        held[b] += 1
                    for at in range(past[b], past[b] + new[b]):
                        slots.append(table[b][at // self.page] * self.page + at % self.page)
                        positions.append(at)
                        requests.append(b)
                else:
                    status[b] = m.REQ_NO_ROOM
            indptr.append(len(slots))
        rest = [-1] * (N - len(slots))
        return dict(indptr=indptr, slots=slots + rest, positions=positions + rest, requests=requests + rest, table=table,
                    held=held, free=free, count=[top], status=status)


def _check(m, s, N, **kw):
    want = s.expected(N, m)
    kept = s.tensors()
    got = m.paged_plan(s.cache_len, s.new_len, s.table, s.held, s.free, s.count, s.page, release=s.release, max_tokens=N,
                       **kw)
    torch.cuda.synchronize()
    for name in ("indptr", "slots", "positions", "requests"):
        t = getattr(got, name)
        assert t.dtype == (torch.int64 if name == "slots" else torch.int32)
        assert t.tolist() == want[name], name
    assert got.req_status.tolist() == want["status"]
    assert s.table.tolist() == want["table"] and s.held.tolist() == want["held"]
    assert s.free.tolist() == want["free"] and s.count.tolist() == want["count"]
    assert torch.equal(s.cache_len, kept[4]) and torch.equal(s.new_len, kept[5])
    assert bool((s.whole[:, s.table.shape[1]:] == -77).all())
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("page", [1, 8, 24, 128])
@pytest.mark.parametrize("past,new", [([0], [1]), ([0], [0]), ([5], [3]), ([128, 0, 77], [1, 9, 0]),
                                      ([7, 24, 23, 48, 0, 1], [17, 1, 1, 0, 300, 24])])
def test_small(m, page, past, new):
    for N in (sum(new), sum(new) + 13):
        _check(m, State(past, new, page, spare=350), N)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 2, 33, 300, 512, 513, 1024, 1500, 4095, 5000, 16384])
def test_many_requests(m, B):
    r = random.Random(B)
    past = [r.randrange(0, 60) for _ in range(B)]
    released = [r.randrange(1, 9) if r.random() < 0.2 else 0 for _ in range(B)]
    past = [0 if x else p for p, x in zip(past, released)]
    new = [r.choice([0, 1, 3, 9, 20]) for _ in range(B)]
    extra = [r.randrange(0, 2) for _ in range(B)]
    s = State(past, new, 8, released=released, extra=extra, spare=4 * B, width=12, stride=3, seed=B)
    _check(m, s, sum(new) + 7)
    _check(m, s, sum(new))     # the same again: former places given back once more, nothing else needed


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[30000], [5000, 0, 8192, 1], [700] * 40])
def test_long_prompts(m, new):
    _check(m, State([0] * len(new), new, 16, spare=2200), sum(new))


@pytest.mark.gpu
def test_pages_given_back_are_taken_in_the_same_call(m):
    """Nothing is free but what two requests give back; one of them is its own successor."""
    s = State([0, 40, 0, 3], [20, 30, 50, 1], 8, released=[6, 0, 9, 0], spare=0)
    got = _check(m, s, 101)
    assert not got.req_status.any() and int(s.count) == 15 - 3 - 4 - 7


@pytest.mark.gpu
@pytest.mark.parametrize("spare", range(0, 12))
def test_a_pool_that_runs_short(m, spare):
    """First come first served, in order: what does not fit holds its place, requests that need nothing go on."""
    s = State([8, 3, 16, 0, 5], [9, 2, 20, 4, 3], 8, spare=spare)
    got = _check(m, s, 38)
    if spare == 3:
        assert got.req_status.tolist() == [0, 0, m.REQ_NO_ROOM, m.REQ_NO_ROOM, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("N", range(0, 12))
def test_a_step_that_has_too_few_rows(m, N):
    _check(m, State([8, 3, 16, 0], [3, 2, 5, 1], 8, spare=20), N)


@pytest.mark.gpu
def test_lengths_that_cannot_be(m):
    s = State([5, 6, 7, 8, 9, 10, 0], [1, 2, 3, 4, 5, 6, 7], 8, width=6, released=[0] * 6 + [4], spare=30)
    s.cache_len[0] = -1
    s.cache_len[1] = 9            # more than the page held
    s.new_len[2] = -3
    s.new_len[3] = 41             # past the table
    s.held[4] = -2
    s.held[5] = 7
    s.cache_len[6] = 3            # the place was given back, its new occupant has nothing cached
    got = _check(m, s, 30)
    assert got.req_status.tolist() == [m.REQ_BAD_LEN] * 7
    s = State([5], [1 << 30], 8, width=6)
    s.cache_len[0] = (1 << 31) - 1
    assert _check(m, s, 4).req_status.tolist() == [m.REQ_BAD_LEN]


@pytest.mark.gpu
@pytest.mark.parametrize("count", [-1, 1000, 1 << 30, -(1 << 31)])
def test_a_pool_that_cannot_be(m, count):
    s = State([5, 6], [1, 20], 8, released=[0, 3], spare=30)
    s.cache_len[1] = 0
    s.count[0] = count
    before = s.tensors()
    got = m.paged_plan(s.cache_len, s.new_len, s.table, s.held, s.free, s.count, 8, release=s.release, max_tokens=9)
    assert all(torch.equal(x, y) for x, y in zip(s.tensors(), before))
    assert got.req_status.tolist() == [m.REQ_BAD_PAGE] * 2
    assert got.indptr.tolist() == [0, 0, 0] and got.slots.tolist() == [-1] * 9


@pytest.mark.gpu
def test_more_pages_given_back_than_the_pool_holds(m):
    """A place that gives back pages which are on the pool already: the pool stays within its bounds."""
    s = State([0, 0], [0, 0], 8, released=[5, 5], spare=3)
    s.count[0] = 12               # of 13 entries
    canary = torch.full((64,), -3, dtype=torch.int32, device="cuda")
    canary[:13] = s.free
    got = m.paged_plan(s.cache_len, s.new_len, s.table, s.held, canary[:13], s.count, 8, release=s.release, max_tokens=1)
    assert int(s.count) == 13 and bool((canary[13:] == -3).all())
    assert got.req_status.tolist() == [m.REQ_BAD_PAGE] * 2


@pytest.mark.gpu
def test_bad_entries_among_the_pages_held(m):
    s = State([20, 9], [2, 1], 8, spare=4)
    s.table[0, 2] = -4
    got = m.paged_plan(s.cache_len, s.new_len, s.table, s.held, s.free, s.count, 8, max_tokens=3)
    assert got.req_status.tolist() == [m.REQ_BAD_PAGE, 0]
    assert got.slots.tolist() == [-1, -1, int(s.table[1, 1]) * 8 + 1] and got.positions.tolist() == [20, 21, 9]


@pytest.mark.gpu
def test_slots_past_32_bits(m):
    s = State([0], [3], 1 << 20, spare=3, width=4)
    s.free[:3] = torch.tensor([4000, 2047, 4096], dtype=torch.int32)
    got = m.paged_plan(s.cache_len, s.new_len, s.table, s.held, s.free, s.count, 1 << 20, max_tokens=3)
    assert got.slots.tolist() == [(4096 << 20) + i for i in range(3)]


@pytest.mark.gpu
def test_no_requests(m):
    i32 = dict(dtype=torch.int32, device="cuda")
    out = m.PagedPlanOutput(torch.full((1,), 7, **i32), torch.full((5,), 7, dtype=torch.int64, device="cuda"),
                            torch.full((5,), 7, **i32), torch.full((5,), 7, **i32), torch.zeros(0, **i32))
    none, count = torch.zeros(0, **i32), torch.tensor([3], **i32)
    m.paged_plan(none, none, torch.zeros(0, 4, **i32), none, torch.arange(3, **i32), count, 16, out=out)
    assert out.indptr.tolist() == [0] and int(count) == 3
    for t in (out.slots, out.positions, out.requests):
        assert t.tolist() == [-1] * 5


@pytest.mark.gpu
def test_outputs_not_wanted_on_another_stream_and_captured(m):
    s = State([5, 6], [3, 20], 8, spare=9, width=8)
    want = s.expected(23, m)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = m.PagedPlanOutput(torch.zeros(3, dtype=torch.int32, device="cuda"), None, None, None,
                            torch.zeros(2, dtype=torch.int32, device="cuda"))
    before = s.tensors()
    m.paged_plan(s.cache_len, s.new_len, s.table, s.held, s.free, s.count, 8, max_tokens=23, out=out, stream=st)
    st.synchronize()
    assert out.indptr.tolist() == want["indptr"] and s.table.tolist() == want["table"]
    for x, y in zip((s.whole, s.held, s.free, s.count), before):
        x.copy_(y)
    out = m.paged_plan(s.cache_len, s.new_len * 0, s.table, s.held, s.free, s.count, 8, max_tokens=23)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.paged_plan(s.cache_len, s.new_len, s.table, s.held, s.free, s.count, 8, out=out)
        s.cache_len += s.new_len
    left = int(s.count)
    past = [5, 6]
    for step in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert out.positions.tolist() == [past[0] + i for i in range(3)] + [past[1] + i for i in range(20)]
        past = [past[0] + 3, past[1] + 20]
        assert s.held.tolist() == [-(-p // 8) for p in past]
        assert int(s.count) == left - (sum(s.held.tolist()) - 2)
    assert not out.req_status.any()


# ------------------------------------------------------------------ the bounds-checked library

@pytest.mark.gpu
@pytest.mark.parametrize("B,N", [(1, 5), (40, 300), (700, 5000), (5000, 9000)])
def test_no_index_of_a_plan_leaves_its_buffer(B, N):
    import test_paged_checked as small
    from speculative_decoding_logit_gb300 import _binding, nvcc_build
    lib = C.CDLL(nvcc_build.build_checked())
    _binding._declare(lib)
    r = random.Random(B)
    released = [r.randrange(1, 9) if r.random() < 0.3 else 0 for _ in range(B)]
    past = [0 if x else r.randrange(0, 60) for x in released]
    s = State(past, [r.choice([0, 1, 3, 9]) for _ in range(B)], 8, released=released, spare=B // 2, width=12, seed=B)
    want = s.expected(N, _binding)
    g = {k: small.Guarded(x) for k, x in dict(table=s.whole, held=s.held, free=s.free, count=s.count).items()}
    i32 = dict(dtype=torch.int32, device="cuda")
    for k, n in dict(indptr=B + 1, positions=N, requests=N, status=B).items():
        g[k] = small.Guarded(torch.zeros(n, **i32))
    g["slots"] = small.Guarded(torch.zeros(N, dtype=torch.int64, device="cuda"))
    at = {k: x.t.data_ptr() for k, x in g.items()}
    pool = _binding._PagePoolC(at["table"], 12, 12, 8, at["held"], at["free"], s.free.numel(), at["count"])
    assert lib.paged_plan(s.cache_len.data_ptr(), s.new_len.data_ptr(), B, C.addressof(pool),
                          s.release.data_ptr() if s.release is not None else None, N, at["indptr"], at["slots"],
                          at["positions"], at["requests"], at["status"], torch.cuda.current_stream().cuda_stream) == 0
    log = (C.c_uint32 * 2)(9, 9)
    assert lib.asv_paged_plan_check_log(log) == 0
    assert list(log) == [0, 0]
    assert all(x.intact() for x in g.values())
    for k, x in g.items():
        assert x.t.tolist() == want[k], k
