"""A decoding step from plan to verification without the host: pages planned, tokens appended with positions of three axes and
attended to, drafts and their distribution sampled into RAPID's tensors, verified, lengths advanced; eager and captured.  The
caches end as one pass over each text leaves them."""
import pytest
import torch

from paged_util import rotation_table

pytestmark = pytest.mark.gpu
VOCAB, Q, KV, DIM, PAGE, B, K, LIMIT = 1003, 4, 2, 32, 8, 5, 3, 400


class Step:
    def __init__(self, asv, seed=0):
        self.asv = asv
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
        self.qkv = rand(VOCAB, (Q + 2 * KV) * DIM).bfloat16()
        self.draft_head = (rand(Q * DIM, VOCAB) * 0.4).bfloat16()
        self.head = (self.draft_head.float() + 0.1 * rand(Q * DIM, VOCAB)).bfloat16()
        self.rotary = rotation_table(LIMIT, DIM).cuda()
        self.axes = bytes([0, 1, 2, 1] * (DIM // 8))
        pages = 2 * B * LIMIT // PAGE
        i32 = dict(dtype=torch.int32, device="cuda")
        self.k_cache, self.v_cache = (torch.zeros(pages, PAGE, KV, DIM, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        self.table = torch.full((B, LIMIT // PAGE), -1, **i32)
        self.held, self.cache_len = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.free = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(**i32)
        self.count = torch.tensor([pages], **i32)
        self.release = torch.zeros(B, dtype=torch.bool, device="cuda")
        self.new_len = torch.full((B,), K + 1, **i32)
        self.one = torch.arange(B + 1, **i32)
        self.last = torch.arange(B, **i32) + 7
        self.u = torch.zeros(B, K + 1, device="cuda")
        self.q = torch.zeros(B, K + 1, VOCAB, device="cuda")
        self.drafts = torch.zeros(B, K + 1, **i32)
        self.status = torch.zeros(B, **i32)
        n = B * (K + 1)
        self.plan = asv.PagedPlanOutput(torch.zeros(B + 1, **i32), torch.zeros(n, dtype=torch.int64, device="cuda"),
                                        torch.zeros(n, **i32), torch.zeros(n, **i32), self.status)
        self.room = torch.zeros(asv.workspace_bytes(asv.ASV_MODE_RAPID, B, K, VOCAB, asv.ASV_F32), dtype=torch.uint8,
                                device="cuda")
        self.attend = torch.zeros(asv.paged_workspace_bytes(Q, KV, DIM), dtype=torch.uint8, device="cuda")
        self.tokens = torch.zeros(B, K + 1, **i32)
        self.accepted = torch.zeros(B, **i32)

    def places(self, at):
        """Axes of time, rows and columns of a position (a page of text four wide)."""
        return torch.stack([at, at.clamp(min=0) // 4, at.clamp(min=0) % 4 + at.clamp(min=0) // 8])

    def forward(self, tokens, at, past, indptr, head):
        q, k, v = self.qkv[tokens.long()].split([Q * DIM, KV * DIM, KV * DIM], 1)
        q, k, v = (x.unflatten(1, (-1, DIM)) for x in (q, k, v))
        app = self.asv.paged_kv_append(k, v, self.k_cache, self.v_cache, self.table, past, indptr, q=q, rotary=self.rotary,
                                       positions=self.places(at), axes=self.axes)
        att = self.asv.paged_attention(app.q, self.k_cache, self.v_cache, self.table, past, indptr, workspace=self.attend)
        self.status |= app.req_status | att.req_status
        return (att.out.flatten(1) @ head).float()

    def step(self):
        asv = self.asv
        asv.paged_plan(self.cache_len, self.new_len, self.table, self.held, self.free, self.count, PAGE, release=self.release,
                       out=self.plan)
        token = self.last
        for i in range(K + 1):  # (the last one for its distribution alone)
            logits = self.forward(token, self.cache_len + i, self.cache_len + i, self.one, self.draft_head)
            asv.sample_tokens(logits, self.u[:, i], temperature=0.8, top_p=0.95,
                              out=asv.SampleOutput(self.drafts[:, i], None, self.q[:, i], self.status))
            token = self.drafts[:, i]
        rows = torch.cat([self.last[:, None], self.drafts[:, :K]], 1)
        z = self.forward(rows.flatten(), self.plan.positions, self.cache_len, self.plan.indptr, self.head)
        out = asv.rapid_verify(z.view(B, K + 1, VOCAB), self.q, self.drafts[:, :K].contiguous(), 1.0, 2.0, 0.1, 5,
                               workspace=self.room)
        self.status |= out.req_status
        self.tokens.copy_(out.tokens)
        self.accepted.copy_(out.accept_len)
        self.cache_len += out.accept_len + 1
        self.last.copy_(out.tokens.gather(1, out.accept_len.long()[:, None])[:, 0])


def _run(s, steps, replay=None):
    """Texts of all requests that were there, and where each ended: (tokens in the cache, table row, place)."""
    u = torch.rand(steps, B, K + 1, generator=torch.Generator().manual_seed(3))
    texts, ended = [[int(t)] for t in s.last.tolist()], []
    for i in range(steps):
        s.u.copy_(u[i])
        s.release.zero_()
        if i == steps // 2:      # one request ends, another takes its place
            texts[2] = [11]
            s.release[2], s.cache_len[2], s.last[2] = True, 0, 11
        replay() if replay else s.step()
        for b in range(B):
            texts[b] += [t for t in s.tokens[b].tolist() if t >= 0]
    torch.cuda.synchronize()
    assert not s.status.any()
    return texts


@pytest.fixture(scope="module")
def asv():
    import speculative_decoding_logit_gb300 as m
    m.build()
    return m


def test_steps_leave_the_caches_as_one_pass_over_the_texts(asv):
    s = Step(asv)
    texts = _run(s, 12)
    lengths, held = s.cache_len.tolist(), s.held.tolist()
    pages = [p for b in range(B) for p in s.table[b, :held[b]].tolist()] + s.free[:int(s.count)].tolist()
    assert sorted(pages) == list(range(s.k_cache.shape[0]))        # every page once
    assert any(a > 0 for a in s.accepted.tolist()) or max(lengths) > 12
    fresh = Step(asv)
    fresh.new_len.copy_(s.cache_len)
    plan = asv.paged_plan(fresh.cache_len, fresh.new_len, fresh.table, fresh.held, fresh.free, fresh.count, PAGE,
                          max_tokens=sum(lengths))
    text = torch.tensor(sum((t[:n] for t, n in zip(texts, lengths)), []), dtype=torch.int32, device="cuda")
    assert all(len(t) == n + 1 for t, n in zip(texts, lengths))     # the last token is not in the cache yet
    fresh.forward(text, plan.positions, fresh.cache_len, plan.indptr, fresh.head)
    for b, n in enumerate(lengths):
        assert held[b] * PAGE >= n
        for c, f in ((s.k_cache, fresh.k_cache), (s.v_cache, fresh.v_cache)):
            at = lambda x, t: x[t[b, :-(-n // PAGE)].long()].flatten(0, 1)[:n]
            assert torch.equal(at(c, s.table), at(f, fresh.table)), b
    slots = plan.slots.cpu()
    assert torch.equal(slots, torch.cat([fresh.table[b, torch.arange(n) // PAGE].cpu().long() * PAGE + torch.arange(n) % PAGE
                                         for b, n in enumerate(lengths)]))
    assert plan.requests.tolist() == [b for b, n in enumerate(lengths) for _ in range(n)]


def test_a_captured_step_is_the_eager_one(asv):
    eager = Step(asv)
    want = _run(eager, 9)
    s = Step(asv)
    first = [t.clone() for t in (s.table, s.held, s.cache_len, s.free, s.count, s.last)]
    s.step()                       # (kernels are loaded before the capture)
    torch.cuda.synchronize()
    for t, v in zip((s.table, s.held, s.cache_len, s.free, s.count, s.last), first):
        t.copy_(v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.step()
    for t, v in zip((s.table, s.held, s.cache_len, s.free, s.count, s.last), first):
        t.copy_(v)
    s.k_cache.zero_()
    s.v_cache.zero_()
    assert _run(s, 9, g.replay) == want
    for a, b in ((s.k_cache, eager.k_cache), (s.v_cache, eager.v_cache), (s.table, eager.table), (s.held, eager.held),
                 (s.free, eager.free), (s.count, eager.count), (s.cache_len, eager.cache_len), (s.q, eager.q)):
        assert torch.equal(a, b)
