"""sample_tokens against the definition in 64 bits (tests/sample_util.py): tokens equal, log-probabilities and distributions
within their bounds; ties, masks, empty nuclei, flat rows, strides, alignment, streams, graphs, refusals."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import test_paged_refusals as host
from sample_util import logprob_bound, off, probs_bound, sample64

NULL, SHAPE, ALIGN, DTYPE, PARAM = 1, 2, 3, 4, 5
m = host.m
BF, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ refusals, on the host

def _call(m, x=None, u=None, one=None, each=None, tokens=None, logprobs=None, probs=None, status=None):
    ref = lambda s: None if s is None else C.addressof(s)
    x, one = x or _logits(m), one or m._SamplingC(1.0, 0, 1.0, 0.0)
    return m.library().sample_tokens(ref(x), ref(u), ref(one), ref(each), ref(tokens), ref(logprobs), ref(probs), status,
                                     None)


def _logits(m, **kw):
    a = dict(data=None, dtype=0, B=2, n=3, V=100, stride_request=300, stride_position=100)
    a.update(kw)
    return m._LogitsC(**a)


def test_sizes(m):
    for kw in (dict(B=-1), dict(n=-1), dict(V=0), dict(V=(1 << 19) + 1), dict(stride_request=-1),
               dict(stride_position=-100), dict(B=1 << 20, n=1 << 10)):
        assert _call(m, _logits(m, **kw)) == SHAPE
    assert _call(m, _logits(m, dtype=2)) == DTYPE
    assert _call(m, _logits(m, B=0)) == 0 and _call(m, _logits(m, n=0)) == 0
    assert _call(m, _logits(m, stride_request=0, stride_position=0)) == NULL   # one row for all
    assert _call(m, _logits(m, B=1, n=1, stride_request=-7, stride_position=-7)) == NULL


@pytest.mark.parametrize("b,n,ok", [(300, 100, True), (100, 200, True), (299, 100, False), (300, 99, False),
                                    (0, 100, False), (-300, 100, False), (100, 199, False), (1000, 0, False)])
def test_rows_that_are_written_are_apart(m, b, n, ok):
    assert _call(m, probs=m._FieldC(None, b, n)) == (NULL if ok else SHAPE)
    small = m._FieldC(None, b // 100 if b % 100 == 0 else b // 100, n // 100)
    if b % 100 == 0 and n % 100 == 0:
        for name in ("tokens", "logprobs"):
            assert _call(m, **{name: small}) == (NULL if ok else SHAPE)


@pytest.mark.parametrize("one", [(-1.0, 0, 1.0, 0.0), (math.nan, 0, 1.0, 0.0), (math.inf, 0, 1.0, 0.0),
                                 (1e-20, 0, 1.0, 0.0), (1e20, 0, 1.0, 0.0), (1.0, -1, 1.0, 0.0), (1.0, 0, 1.01, 0.0),
                                 (1.0, 0, -0.1, 0.0), (1.0, 0, math.nan, 0.0), (1.0, 0, 1.0, -0.1),
                                 (1.0, 0, 1.0, 1.5), (1.0, 0, 1.0, math.nan)])
def test_parameters(m, one):
    assert _call(m, one=m._SamplingC(*one)) == PARAM
    each = m._SamplingEachC(*[host.BASE] * 4)            # the requests' own stand in for all four
    assert _call(m, one=m._SamplingC(*one), each=each) == NULL


def test_alignment_and_pointers(m):
    odd = host.BASE + 2
    assert _call(m, _logits(m, data=odd)) == ALIGN
    assert _call(m, _logits(m, data=odd, dtype=1)) == NULL
    assert _call(m, _logits(m, data=odd + 1, dtype=1)) == ALIGN
    for name in ("u", "tokens", "logprobs"):
        assert _call(m, **{name: m._FieldC(odd, 3, 1)}) == ALIGN
    assert _call(m, probs=m._FieldC(odd, 300, 100)) == ALIGN
    for i in range(4):
        assert _call(m, each=m._SamplingEachC(*[odd if i == j else None for j in range(4)])) == ALIGN
    assert _call(m, status=odd) == ALIGN
    assert _call(m) == NULL
    assert m.library().sample_tokens(*[None] * 9) == NULL


def test_binding_refuses_host_tensors(m):
    with pytest.raises(m.AsvError):
        m.sample_tokens(torch.zeros(1, 8), torch.zeros(1))


@pytest.mark.gpu
def test_binding_refuses_shapes_and_types(m):
    x, u = torch.zeros(2, 3, 50, device="cuda"), torch.zeros(2, 3, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")

    def status(x=x, u=u, **kw):
        with pytest.raises(m.AsvError) as e:
            m.sample_tokens(x, u, **kw)
        return e.value.status

    def out(**kw):
        o = m.SampleOutput(torch.zeros(2, 3, **i32), torch.zeros(2, 3, device="cuda"), None, torch.zeros(2, **i32))
        for k, v in kw.items():
            setattr(o, k, v)
        return o

    assert status(x.half()) == DTYPE
    assert status(x.double()) == DTYPE
    assert status(x[0, 0]) == SHAPE
    assert status(x[None]) == SHAPE
    assert status(x.transpose(1, 2).contiguous().transpose(1, 2)) == SHAPE
    assert status(x[:, :, :0]) == SHAPE
    assert status(u=u[:, :2]) == SHAPE
    assert status(u=u[0]) == SHAPE
    assert status(u=u.double()) == DTYPE
    assert status(u=u.cpu()) == -1
    assert status(temperature=torch.ones(3, device="cuda")) == SHAPE
    assert status(temperature=torch.ones(2, **i32)) == DTYPE
    assert status(top_k=torch.ones(2, device="cuda")) == DTYPE
    assert status(temperature=None) == PARAM
    assert status(top_k=1.5) == PARAM
    assert status(top_k=-1) == PARAM
    assert status(top_p=1.5) == PARAM
    assert status(temperature=-1.0) == PARAM
    assert status(out=out(tokens=torch.zeros(2, 3, dtype=torch.int64, device="cuda"))) == DTYPE
    assert status(out=out(tokens=torch.zeros(2, 2, **i32))) == SHAPE
    assert status(out=out(tokens=torch.zeros(2, 1, **i32).expand(2, 3))) == SHAPE
    assert status(out=out(probs=torch.zeros(2, 3, 49, device="cuda"))) == SHAPE
    assert status(out=out(probs=torch.zeros(2, 3, 50, dtype=BF, device="cuda"))) == DTYPE
    assert status(out=out(probs=torch.zeros(2, 1, 50, device="cuda").expand(2, 3, 50))) == SHAPE
    assert status(out=out(req_status=None)) == NULL
    assert status(out=out(req_status=torch.zeros(3, **i32))) == SHAPE


# ------------------------------------------------------------------ results

def _compare(x, u, got, T, k, p, least, probs=True):
    """x and u on the host; parameters: numbers or lists, one to a request."""
    each = lambda v, b: v[b] if isinstance(v, (list, tuple)) else v
    f32 = lambda v: float(np.float32(v))
    B, n, V = x.shape
    left = 0
    for b in range(B):
        for i in range(n):
            token, lp, dist, margin = sample64(x[b, i].double().numpy(), float(u[b, i]), f32(each(T, b)), each(k, b),
                                               f32(each(p, b)), f32(each(least, b)))
            if margin < 1:
                left += 1
                continue
            assert int(got.tokens[b, i]) == token, (b, i, margin)
            assert abs(float(got.logprobs[b, i]) - lp) <= logprob_bound(lp), (b, i, float(got.logprobs[b, i]), lp)
            if probs:
                have = got.probs[b, i].double().cpu().numpy()
                far = np.abs(have - dist) > probs_bound(dist)
                assert not far.any(), (b, i, int(far.argmax()), have[far][0], dist[far][0])
    assert left <= 1 + B * n // 50   # (of 50 thousand borders one is that near in 2e-4 of the rows)
    assert not got.req_status.any()


def _logits_of(B, n, V, kind, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "peaked":
        x = -1.5 * torch.empty(B, n, V).exponential_(generator=g).log() + 1.1 * torch.empty(B, n, V).exponential_(generator=g)
    elif kind == "flat":
        x = 2 * torch.randn(B, n, V, generator=g)
    elif kind == "ties":
        x = torch.randint(-3, 4, (B, n, V), generator=g).float()
    elif kind == "masked":
        x = 3 * torch.randn(B, n, V, generator=g)
        x[torch.rand(B, n, V, generator=g) < 0.6] = -math.inf
        x[torch.rand(B, n, V, generator=g) < 0.2] = torch.finfo(dtype).min
        x[:, :, V // 2] = 1.0
    elif kind == "equal":
        x = torch.full((B, n, V), -7.25)
    elif kind == "negative":
        x = -100 - 5 * torch.rand(B, n, V, generator=g)
    return x.to(dtype)


def _draws(B, n, seed=0):
    return torch.rand(B, n, generator=torch.Generator().manual_seed(1000 + seed))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 33, 1001, 4099, 20000])
@pytest.mark.parametrize("kind", ["peaked", "flat", "ties", "masked", "equal", "negative"])
def test_kinds_of_rows(m, dtype, V, kind):
    B, n = 3, 2
    x, u = _logits_of(B, n, V, kind, dtype, V), _draws(B, n, V)
    for T, k, p, least in ((1.0, 0, 1.0, 0.0), (0.7, 40, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.3, 0, 1.0, 0.1),
                           (0.8, 5, 0.95, 0.05), (0.0, 3, 0.5, 0.0), (1.0, 1, 1.0, 0.0), (1.0, 0, 0.0, 0.0),
                           (1.0, 2000, 0.99, 0.0), (1.0, 0, 1.0, 1.0), (20.0, 0, 0.999, 1e-6)):
        got = m.sample_tokens(x.cuda(), u.cuda(), temperature=T, top_k=k, top_p=p, min_p=least, probs=True)
        _compare(x, u, got, T, k, p, least)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["peaked", "flat", "ties"])
@pytest.mark.parametrize("B", [1, 3, 30])
def test_large_vocabularies(m, dtype, kind, B):
    V = 151936
    x, u = _logits_of(B, 1, V, kind, dtype, B), _draws(B, 1, B)
    for T, k, p, least in ((1.0, 0, 1.0, 0.0), (0.8, 50, 0.95, 0.0), (0.9, 0, 0.9, 0.0), (1.0, 3000, 0.99, 0.0)):
        got = m.sample_tokens(x.cuda(), u.cuda(), temperature=T, top_k=k, top_p=p, min_p=least, probs=B == 3)
        _compare(x, u, got, T, k, p, least, probs=B == 3)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_parameters_of_each_request(m, dtype):
    B, n, V = 40, 3, 3001
    x, u = _logits_of(B, n, V, "peaked", dtype, 5), _draws(B, n, 5)
    T = [[0.0, 0.5, 1.0, 1.7][i % 4] for i in range(B)]
    k = [[0, 1, 7, 100, 5000][i % 5] for i in range(B)]
    p = [[1.0, 0.3, 0.9][i % 3] for i in range(B)]
    least = [[0.0, 0.01, 0.0, 0.3][i // 4 % 4] for i in range(B)]
    f = lambda v: torch.tensor(v, dtype=F32, device="cuda")
    got = m.sample_tokens(x.cuda(), u.cuda(), temperature=f(T), top_k=torch.tensor(k, dtype=torch.int32, device="cuda"),
                          top_p=f(p), min_p=f(least), probs=True)
    _compare(x, u, got, T, k, p, least)
    mixed = m.sample_tokens(x.cuda(), u.cuda(), temperature=f(T), top_k=50, top_p=f(p), min_p=0.0, probs=True)
    _compare(x, u, mixed, T, 50, p, 0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_ends_of_the_draw(m, dtype):
    """u = 0, the last below 1, what is outside [0, 1) and NaN: the first kept token, the last."""
    x = _logits_of(1, 8, 5000, "peaked", dtype, 3)
    u = torch.tensor([[0.0, -0.0, -3.0, math.nan, 0.99999994, 1.0, 7.0, math.inf]])
    for k, p in ((0, 1.0), (20, 1.0), (0, 0.9)):
        got = m.sample_tokens(x.cuda(), u.cuda(), top_k=k, top_p=p, probs=True)
        clipped = torch.tensor([[0.0, 0.0, 0.0, 0.0] + [0.99999994] * 4])
        _compare(x, clipped, got, 1.0, k, p, 0.0)


@pytest.mark.gpu
def test_rare_weights_count(m):
    """A heavy entry over many light ones: the light ones' mass is where half of the draws fall."""
    V = 100001
    x = torch.zeros(1, 64, V)
    x[:, :, 777] = math.log(V - 1)
    x += 0.001 * torch.randn(1, 64, V, generator=torch.Generator().manual_seed(2))
    u = _draws(1, 64, 9)
    for T, k, p, least in ((1.0, 0, 1.0, 0.0), (1.0, 0, 0.75, 0.0), (1.0, 60000, 1.0, 0.0)):
        got = m.sample_tokens(x.cuda(), u.cuda(), temperature=T, top_k=k, top_p=p, min_p=least, probs=True)
        _compare(x, u, got, T, k, p, least)


@pytest.mark.gpu
def test_extreme_values(m):
    big = torch.finfo(F32).max
    rows = [[big, -big, 0.0, big], [1e30, 1e30, 9e29, -math.inf], [-big, -big, -math.inf, -big],
            [1e-45, 0.0, -0.0, -1e-45], [-0.0, 0.0, 0.0, -0.0], [3.0, math.nextafter(3.0, 4.0), 3.0, 2.9999998]]
    x = torch.tensor(rows, dtype=F32)[:, None].repeat(1, 4, 1)
    u = torch.tensor([[0.1, 0.4, 0.6, 0.9]]).repeat(len(rows), 1)
    for T, k, p in ((1.0, 0, 1.0), (1.0, 2, 1.0), (1e-15, 0, 0.9), (1e15, 3, 0.9), (2.0 ** -64, 0, 1.0), (2.0 ** 64, 0, 0.6)):
        got = m.sample_tokens(x.cuda(), u.cuda(), temperature=T, top_k=k, top_p=p, probs=True)
        _compare(x, u, got, T, k, p, 0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_that_are_flagged(m, dtype):
    x = _logits_of(6, 2, 700, "peaked", dtype)
    u = _draws(6, 2)
    x[1, 0, 699] = math.nan
    x[2, 1, 0] = math.inf
    x[3, :] = -math.inf
    x[4, 0, 5] = -math.inf                    # a single one is a probability of 0
    T = [1.0] * 5 + [-1.0]
    got = m.sample_tokens(x.cuda(), u.cuda(), temperature=torch.tensor(T, device="cuda"), top_k=9, probs=True)
    assert got.req_status.tolist() == [0, m.REQ_NONFINITE, m.REQ_NONFINITE, m.REQ_NONFINITE, 0, m.REQ_BAD_PARAM]
    flagged = {(1, 0), (2, 1), (3, 0), (3, 1), (5, 0), (5, 1)}
    for b in range(6):
        for i in range(2):
            if (b, i) in flagged:
                assert int(got.tokens[b, i]) == -1 and float(got.logprobs[b, i]) == -math.inf
                assert not got.probs[b, i].any()
            else:
                assert int(got.tokens[b, i]) == sample64(x[b, i].double().numpy(), float(u[b, i]), 1.0, 9, 1.0, 0.0)[0]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shift", range(0, 8))
def test_strides_and_alignment(m, dtype, shift):
    """Rows at every alignment, every output inside a larger buffer that keeps the rest of what it held."""
    B, n, V = 3, 2, 517
    x, u = _logits_of(B, n, V, "peaked", dtype, shift), _draws(B, n, shift)
    wide = torch.full((n, B, V + 13), math.nan, dtype=dtype, device="cuda")
    wide[:, :, shift:shift + V] = x.transpose(0, 1).cuda()
    uu = torch.rand(n, B, 3, device="cuda")
    uu[:, :, 1] = u.T.cuda()
    tokens, logs = torch.full((B, 5), -9, dtype=torch.int32, device="cuda"), torch.full((n, 7, B), 9.0, device="cuda")
    probs = torch.full((B, 4, V + 9), 9.0, device="cuda")
    out = m.SampleOutput(tokens[:, 1:1 + n], logs[:, 2].T, probs[:, 1:1 + n, shift:shift + V],
                         torch.zeros(B, dtype=torch.int32, device="cuda"))
    m.sample_tokens(wide.transpose(0, 1)[:, :, shift:shift + V], uu.transpose(0, 1)[:, :, 1], top_k=30, top_p=0.9, out=out)
    _compare(x, u, out, 1.0, 30, 0.9, 0.0)
    assert bool((tokens[:, 0] == -9).all()) and bool((tokens[:, 1 + n:] == -9).all())
    logs[:, 2] = 9.0
    probs[:, 1:1 + n, shift:shift + V] = 9.0
    assert bool((logs == 9).all()) and bool((probs == 9).all())


@pytest.mark.gpu
def test_two_dimensions_one_row_for_all_and_positions_in_turn(m):
    V = 900
    x, u = _logits_of(5, 4, V, "peaked", F32, 1), _draws(5, 4, 1)
    whole = m.sample_tokens(x.cuda(), u.cuda(), temperature=0.9, probs=True)
    _compare(x, u, whole, 0.9, 0, 1.0, 0.0)
    # a position at a time into RAPID's tensors
    q, ids = torch.zeros(5, 4, V, device="cuda"), torch.zeros(5, 4, dtype=torch.int32, device="cuda")
    status = torch.zeros(5, dtype=torch.int32, device="cuda")
    for i in range(4):
        m.sample_tokens(x[:, i].cuda(), u[:, i].cuda(), temperature=0.9, out=m.SampleOutput(ids[:, i], None, q[:, i], status))
    assert torch.equal(ids, whole.tokens) and torch.equal(q, whole.probs)
    got = m.sample_tokens(x[:1].cuda().expand(5, 4, V), u.cuda(), top_k=3)
    _compare(x[:1].expand(5, 4, V), u, got, 1.0, 3, 1.0, 0.0, probs=False)
    # nothing to do
    assert m.sample_tokens(x[:0].cuda(), u[:0].cuda()).tokens.shape == (0, 4)
    assert m.sample_tokens(x[:, :0].cuda(), u[:, :0].cuda()).tokens.shape == (5, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_result_does_not_depend_on_the_batch(m, dtype):
    """One row to a cluster of many CTAs and to one: the same token and the same cut (entries that are kept), and numbers
    within twice their bounds of each other."""
    V = 40000
    for kind in ("peaked", "flat"):
        x, u = _logits_of(1, 1, V, kind, dtype, 4).cuda(), _draws(1, 1, 4).cuda()
        for kw in (dict(), dict(top_k=40), dict(top_p=0.9), dict(top_p=0.95, min_p=0.01, temperature=0.6)):
            one = m.sample_tokens(x, u, probs=True, **kw)
            many = m.sample_tokens(x.expand(700, 1, V), u.expand(700, 1), probs=True, **kw)
            assert bool((many.tokens == one.tokens).all())
            lp = float(one.logprobs)
            assert float((many.logprobs - lp).abs().max()) <= 2 * logprob_bound(lp)
            p = one.probs.double()
            assert bool(((many.probs - p).abs() <= 2 * probs_bound(p)).all())
            assert bool(((many.probs > 0) == (one.probs > 0)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("ctas", range(1, 9))
def test_numbers_of_ctas(m, ctas):
    """Rows cut into one to eight runs, the last ones short or empty."""
    m.set_tuning(ctas, 0)
    try:
        for dtype, V, kind in ((BF, 3, "peaked"), (F32, 61, "ties"), (BF, 2047, "peaked"), (F32, 30001, "flat"), (BF, 30001, "ties")):
            x, u = _logits_of(2, 2, V, kind, dtype, ctas), _draws(2, 2, ctas)
            for T, k, p, least in ((1.0, 0, 1.0, 0.0), (0.9, 17, 0.95, 0.0), (1.0, 0, 0.9, 0.0), (0.0, 0, 1.0, 0.0),
                                   (1.0, 1500, 0.9, 0.0), (1.0, 0, 0.99, 0.01)):
                got = m.sample_tokens(x.cuda(), u.cuda(), temperature=T, top_k=k, top_p=p, min_p=least, probs=True)
                _compare(x, u, got, T, k, p, least)
    finally:
        m.set_tuning(0, 0)


@pytest.mark.gpu
def test_on_another_stream_and_captured(m):
    x, u = _logits_of(4, 2, 6000, "peaked", BF, 6), _draws(4, 2, 6)
    xd, ud = x.cuda(), u.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = m.sample_tokens(xd, ud, top_p=0.9, probs=True, stream=s)
    s.synchronize()
    _compare(x, u, got, 1.0, 0, 0.9, 0.0)
    out = m.sample_tokens(xd, ud, top_p=0.9, probs=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.sample_tokens(xd, ud, top_p=0.9, out=out)
    x2, u2 = _logits_of(4, 2, 6000, "flat", BF, 7), _draws(4, 2, 7)
    xd.copy_(x2)
    ud.copy_(u2)
    g.replay()
    torch.cuda.synchronize()
    _compare(x2, u2, out, 1.0, 0, 0.9, 0.0)


@pytest.mark.gpu
def test_frequencies(m):
    """200 thousand draws from one distribution: chi-square over its 16 tokens."""
    x = torch.tensor([0.0, 1.0, -1.0, 2.0, 0.5, -3.0, 1.5, 0.25, -0.5, 3.0, -2.0, 0.75, 1.25, -1.5, 2.5, 0.1])
    rows = 200000
    u = torch.rand(rows, 1, device="cuda", generator=torch.Generator("cuda").manual_seed(11))
    got = m.sample_tokens(x.cuda().expand(rows, 1, 16), u, temperature=1.1)
    p = torch.softmax(x.double() / float(np.float32(1.1)), 0)
    seen = torch.bincount(got.tokens.flatten().cpu().long(), minlength=16).double()
    chi = float(((seen - rows * p) ** 2 / (rows * p)).sum())
    assert chi < 44.0    # 15 degrees of freedom: 44 is passed with probability 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [(77, 1), (40, 5), (1300, 1)])
def test_many_rows(m, dtype, rows):
    """More rows than are taken whole by one launch: settled by the first or left to the one behind it, mixed."""
    B, n, V = *rows, 5003
    x, u = _logits_of(B, n, V, "peaked", dtype, B), _draws(B, n, B)
    flat = torch.arange(B) % 3 == 0
    x[flat] = _logits_of(int(flat.sum()), n, V, "flat", dtype, 1)
    x[1] = 0.5                                         # all equal
    for T, k, p, least in ((1.0, 0, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (0.9, 30, 0.95, 0.02), (1.0, 1500, 0.9, 0.0), (0.0, 0, 1.0, 0.0)):
        got = m.sample_tokens(x.cuda(), u.cuda(), temperature=T, top_k=k, top_p=p, min_p=least, probs=B == 77)
        _compare(x, u, got, T, k, p, least, probs=B == 77)
    x[5, 0, 17], x[6, 0, 3] = math.nan, math.inf
    got = m.sample_tokens(x.cuda(), u.cuda(), top_p=0.9)
    assert got.req_status.nonzero().flatten().tolist() == [5, 6] and int(got.tokens.min()) == -1


def _in_general(V, kind):
    g = torch.Generator().manual_seed(V)
    if kind == "pairs":          # two values next to each other, each many times
        return 1.0 + 1e-4 * torch.randint(0, 2, (V,), generator=g)
    if kind == "steps":          # equal values that a border falls among
        return torch.randint(-40, 0, (V,), generator=g) / 16.0
    if kind == "wide":           # more decades than weights have
        return -200 * torch.rand(V, generator=g)
    return 2 * torch.randn(V, generator=g)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 80])
@pytest.mark.parametrize("kind", ["pairs", "steps", "wide", "flat"])
def test_borders_of_rows_in_general(m, dtype, rows, kind):
    """Rows whose kept set is too large to be listed: borders among equal values, among values that no histogram by value
    tells apart, of a nucleus within a top-k, and min-p's within them."""
    V = 30011
    few = [0, rows // 2, rows - 1][:1 if rows == 1 else 3]
    x = _in_general(V, kind).to(dtype).expand(rows, 1, V).contiguous()
    u = _draws(rows, 1, V)
    for T, k, p, least in ((1.0, 0, 0.5, 0.0), (1.0, 0, 0.97, 0.0), (1000.0, 0, 0.9, 0.0), (1.0, 9000, 1.0, 0.0),
                           (1.0, 20000, 0.6, 0.0), (0.7, 0, 0.9, 0.02), (1000.0, 15000, 1.0, 0.9), (1e-3, 12000, 0.999, 0.0)):
        got = m.sample_tokens(x.cuda(), u.cuda(), temperature=T, top_k=k, top_p=p, min_p=least, probs=True)
        got = m.SampleOutput(*(t.cpu()[few] for t in (got.tokens, got.logprobs, got.probs, got.req_status)))
        _compare(x[few], u[few], got, T, k, p, least)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["flat", "peaked", "ties"])
@pytest.mark.parametrize("V,B", [(20011, 60), (151936, 90)])
def test_draws_next_to_borders(m, dtype, kind, V, B):
    """u at the fp32 number nearest to where one token ends and the next begins, 2^-25 of the mass away at most.  Weights'
    sums may be off by 2^-29 + V 2^-44 of it, 2^-26.7 at 151,936, so a good part of the draws is too near to tell the token;
    theirs may be any that u falls into with that much to both sides (several, where a token's mass is less)."""
    x = _logits_of(1, 1, V, kind, dtype, V)
    for p in (1.0, 0.97):
        y, p32 = x[0, 0].double().numpy(), float(np.float32(p))
        dist = sample64(y, 0.5, 1.0, 0, p32, 0.0)[2]
        upto = np.cumsum(dist)
        at = np.searchsorted(upto, np.random.default_rng(V).uniform(0.001, 0.999, B))
        u = torch.from_numpy(upto[at].astype(np.float32)).view(B, 1).clamp(max=1 - 2 ** -24)
        got = m.sample_tokens(x.expand(B, 1, V).cuda(), u.cuda(), top_p=p)
        assert not got.req_status.any()
        for b in range(20):
            token, lp, _, margin = sample64(y, float(u[b, 0]), 1.0, 0, p32, 0.0)
            have = int(got.tokens[b, 0])
            if margin >= 1:
                assert have == token, (b, margin)
                assert abs(float(got.logprobs[b, 0]) - lp) <= logprob_bound(lp)
            else:
                assert dist[have] > 0, b
                assert upto[have] - dist[have] - off(1.0, V) <= float(u[b, 0]) <= upto[have] + off(1.0, V), (b, margin)
