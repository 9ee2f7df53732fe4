"""Larger paged batches for the tests: what they hold made on the GPU in a few calls, the split of their work worked out
request by request, and their attention in 64 bits, a request and a key head at a time."""
import math

import torch

from paged_util import half_step

TILE = 128


class LongBatch:
    """Like paged_util.Batch (the same names), with the values made on the GPU: every slot that no request has written,
    and the tail of the last page, holds NaN; entries of the block table past a request's last page are out of range."""

    def __init__(self, q_lens, past, *, heads, dim, page=16, dtype=torch.bfloat16, seed=0, gain=1.0):
        self.q_lens, self.past, self.page, self.dtype, self.dim = list(q_lens), list(past), page, dtype, dim
        self.Hq, self.Hkv = heads
        self.group, self.B = heads[0] // heads[1], len(self.q_lens)
        g = torch.Generator(device="cuda").manual_seed(seed)
        need = [-(-(a + n) // page) for a, n in zip(past, q_lens)]
        n_pages = sum(need) + 3
        order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
        self.rows, at = [], 0
        for n in need:
            self.rows.append(order[at:at + n])
            at += n
        width = max(need) + 1
        bad = [-1, n_pages, 1 << 30, -(1 << 31)]
        self.table = torch.tensor([r + [bad[(i + j) % 4] for j in range(width - len(r))] for i, r in enumerate(self.rows)],
                                  dtype=torch.int32, device="cuda")
        self.starts = [0]
        for n in q_lens:
            self.starts.append(self.starts[-1] + n)
        self.N = self.starts[-1]
        self.indptr = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        self.cache_len = torch.tensor(self.past, dtype=torch.int32, device="cuda")
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
        self.k = [(rand(a + n, self.Hkv, dim) * gain).to(dtype) for a, n in zip(past, q_lens)]
        self.v = [rand(a + n, self.Hkv, dim).to(dtype) for a, n in zip(past, q_lens)]
        self.qd = (rand(self.N, self.Hq, dim) * 2 * gain).to(dtype)
        self.n_pages = n_pages

    def fill(self):
        """Writes the requests' tokens to the caches."""
        shape = (self.n_pages, self.page, self.Hkv, self.dim)
        self.k_cache, self.v_cache = (torch.full(shape, math.nan, dtype=self.dtype, device="cuda") for _ in range(2))
        for r, k, v in zip(self.rows, self.k, self.v):
            at = torch.arange(k.shape[0], device="cuda")
            to = torch.tensor(r + [0], device="cuda")[at // self.page], at % self.page
            self.k_cache[to], self.v_cache[to] = k, v
        return self

    def args(self):
        return self.qd, self.k_cache, self.v_cache, self.table, self.cache_len, self.indptr


class Plan:
    """The split of a batch: row tiles of an item (1 or 2), whether the row tile is divided, and the pieces of every CTA,
    (request, key head, first token, tokens, [t0, t1) of the item's key tiles, whole item or not) in order."""

    def __init__(self, b, window=0, ctas=None):
        ctas = ctas or torch.cuda.get_device_properties(0).multi_processor_count
        self.two = b.N * b.group > TILE * b.B
        self.divided = b.N % b.B == 0 and b.N * b.group <= 32 * b.B
        tokens = (32 if self.divided else TILE) // b.group * (2 if self.two else 1)
        cost = 1 if self.divided and b.B * b.Hkv > ctas else 2
        items = []
        for r, (n, a) in enumerate(zip(b.q_lens, b.past)):
            mine = []
            for i in range(0, n, tokens):
                count = min(tokens, n - i)
                lo = max(0, a + i - window + 1) if window else 0
                mine.append((i, count, lo // TILE, -(-(a + i + count) // TILE)))
            items += [(r, h, *it) for it in mine for h in range(b.Hkv)]
        total = sum(t1 - t0 + cost for *_, t0, t1 in items)
        run = -(-total // ctas)
        self.run, self.units = run, total
        cuts = [c * total // ctas if run > 16 else min(c * run, total) for c in range(ctas + 1)]
        self.pieces = [[] for _ in range(ctas)]
        at, c = 0, 0
        for r, h, i, count, t0, t1 in items:
            n, first = t1 - t0, at + cost
            while c < ctas and cuts[c + 1] <= at:
                c += 1
            k = c
            while k < ctas and cuts[k] < first + n:
                x, y = max(cuts[k], first), min(cuts[k + 1], first + n)
                if x < y:
                    self.pieces[k].append((r, h, i, count, t0 + x - first, t0 + y - first, y - x == n))
                k += 1
            at += n + cost

    def all(self):
        return [p for ps in self.pieces for p in ps]

    def longest(self):
        """Key tiles of the longest piece, whole and cut."""
        return tuple(max([y - x for *_, x, y, w in self.all() if w == whole], default=0) for whole in (True, False))


def attention64_wide(b, scale=None, window=0, requests=None):
    """{request: (out, lse, out's bound, lse's bound)} in 64 bits on the GPU, for all requests or those given; the bounds
    are paged_util.attention64's, but that fp16 weights lose at most 2^-32 (half the smallest step, 2^-25, next to weights
    whose largest is at least 2^7)."""
    D, G = b.dim, b.group
    scale = D ** -0.5 if scale is None else scale
    u = half_step(b.dtype)
    tiny = 2.0 ** -32 if b.dtype == torch.float16 else 0.0
    res = {}
    for r in range(b.B) if requests is None else requests:
        n, a = b.q_lens[r], b.past[r]
        if not n:
            continue
        pos = a + torch.arange(n, device="cuda").repeat_interleave(G)[:, None]
        key = torch.arange(a + n, device="cuda")[None]
        seen = key <= pos
        if window:
            seen &= key > pos - window
        keys = seen.sum(1, keepdim=True)
        outs = []
        for h in range(b.Hkv):
            k, v = b.k[r][:, h].double(), b.v[r][:, h].double()
            q = b.qd[b.starts[r]:b.starts[r + 1], h * G:(h + 1) * G].double().reshape(n * G, D)
            s = (q @ k.T * scale).masked_fill(~seen, -math.inf)
            top = s.abs().masked_fill(~seen, 0).amax(-1, keepdim=True)
            size = (q.abs() @ k.abs().T * scale).masked_fill(~seen, 0).amax(-1, keepdim=True)
            lse = torch.logsumexp(s, -1, keepdim=True)
            p = torch.exp(s - lse)
            o, weight = p @ v, p @ v.abs()
            ds = size * (D + 2) * 2.0 ** -24 + top * 2.0 ** -23 + 2.0 ** -20
            rel = u + 2 * ds + (keys + D) * 2.0 ** -23
            tol = u * o.abs() + weight * rel * (1 + u) + tiny * (1 + seen.double() @ v.abs())
            ltol = ds + keys * 2.0 ** -23 + 2.0 ** -22 * (1 + lse.abs())
            outs.append([x.reshape(n, G, -1) for x in (o, lse, tol, ltol)])
        o, lse, tol, ltol = (torch.cat(x, 1) for x in zip(*outs))
        res[r] = o, lse[..., 0], tol, ltol[..., 0]
    return res


def assert_requests(b, got, want, what=""):
    for r, (o, lse, tol, ltol) in want.items():
        rows = slice(b.starts[r], b.starts[r + 1])
        for x, y, t, name in ((got.out[rows], o, tol, "out"), (got.lse[rows], lse, ltol, "lse")):
            bad = ~((x.double() - y).abs() <= t)
            if bool(bad.any()):
                at = tuple(int(i) for i in bad.nonzero()[0])
                raise AssertionError(f"{what}{name} of request {r}: {int(bad.sum())} of {bad.numel()} outside; first at {at}: "
                                     f"{float(x[at])} against {float(y[at])}, allowed {float(t[at])}")
