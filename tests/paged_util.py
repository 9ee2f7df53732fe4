"""Paged-cache batches for the tests, and what the operators compute on them in 64 bits, with the error
bounds that the kernels' roundings allow."""
import math

import torch


def half_step(dtype):
    """The largest relative error of one rounding to `dtype`."""
    return torch.finfo(dtype).eps / 2


class Batch:
    """A batch of chunks over a paged cache.  Every slot that no request has written, and the tail of
    the last page, holds NaN; entries of the block table past a request's last page are out of range."""

    def __init__(self, q_lens, past, *, heads=(4, 2), dim=64, page=16, dtype=torch.bfloat16, heads_first=False,
                 seed=0, device="cuda", gain=1.0, spare_pages=3):
        self.q_lens, self.past, self.page, self.dtype, self.dim = list(q_lens), list(past), page, dtype, dim
        self.Hq, self.Hkv = heads
        self.group = self.Hq // self.Hkv
        g = torch.Generator().manual_seed(seed)
        need = [-(-(a + n) // page) for a, n in zip(past, q_lens)]
        n_pages = sum(need) + spare_pages
        order = torch.randperm(n_pages, generator=g).tolist()
        self.rows, at = [], 0
        for n in need:
            self.rows.append(order[at:at + n])
            at += n
        width = max(need + [1]) + 1
        bad = [-1, n_pages, 1 << 30, -(1 << 31)]
        self.table = torch.tensor([r + [bad[(i + j) % 4] for j in range(width - len(r))]
                                   for i, r in enumerate(self.rows)], dtype=torch.int32, device=device)
        starts = [0]
        for n in q_lens:
            starts.append(starts[-1] + n)
        self.starts = starts
        self.N = starts[-1]
        self.indptr = torch.tensor(starts, dtype=torch.int32, device=device)
        self.cache_len = torch.tensor(past, dtype=torch.int32, device=device)
        B = len(q_lens)
        # what each request holds, in order
        self.k = [(torch.randn(a + n, self.Hkv, dim, generator=g) * gain).to(dtype) for a, n in zip(past, q_lens)]
        self.v = [torch.randn(a + n, self.Hkv, dim, generator=g).to(dtype) for a, n in zip(past, q_lens)]
        self.q = (torch.randn(self.N, self.Hq, dim, generator=g) * 2 * gain).to(dtype)
        shape = (n_pages, self.Hkv, page, dim) if heads_first else (n_pages, page, self.Hkv, dim)
        self.k_cache, self.v_cache = (torch.full(shape, math.nan, dtype=dtype) for _ in range(2))
        if heads_first:
            self.k_cache, self.v_cache = self.k_cache.transpose(1, 2), self.v_cache.transpose(1, 2)
        self.B = B

    def fill(self, upto=None):
        """Writes the requests' tokens (all, or the first `upto[b]`) to the caches; returns self on the GPU."""
        for b, r in enumerate(self.rows):
            n = self.past[b] + self.q_lens[b] if upto is None else upto[b]
            for j in range(n):
                self.k_cache[r[j // self.page], j % self.page] = self.k[b][j]
                self.v_cache[r[j // self.page], j % self.page] = self.v[b][j]
        self.k_cache, self.v_cache, self.qd = self.k_cache.cuda(), self.v_cache.cuda(), self.q.cuda()
        return self

    def new_rows(self):
        """The chunks' keys and values, packed."""
        k = [self.k[b][self.past[b]:] for b in range(self.B)]
        v = [self.v[b][self.past[b]:] for b in range(self.B)]
        return torch.cat(k), torch.cat(v)


def attention64(batch, scale=None, window=0):
    """(out, lse, out's bound, lse's bound) in 64 bits.

    Bounds: the scores are sums of D exact products in fp32, in any order, then one product with the
    scale (ds); exp2's argument and value add 2^-20 at most for |s| < 64 (the argument's rounding, half a
    step of |s| log2 e, and the special-function unit's); each weight is rounded once to the cache's type
    (u; fp16 also loses up to half its smallest step, 2^-25, next to weights whose largest is at least 1);
    n terms are summed in fp32; out is rounded once."""
    D = batch.dim
    scale = D ** -0.5 if scale is None else scale
    u = half_step(batch.dtype)
    tiny = 2.0 ** -25 if batch.dtype == torch.float16 else 0.0
    outs, lses, tols, ltols = [], [], [], []
    for b in range(batch.B):
        n, a = batch.q_lens[b], batch.past[b]
        k, v = batch.k[b].double(), batch.v[b].double()
        q = batch.q[batch.starts[b]:batch.starts[b + 1]].double()
        for i in range(n):
            lo = max(0, a + i + 1 - window) if window else 0
            kk = k[lo:a + i + 1].repeat_interleave(batch.group, 1)   # [n_keys, Hq, D]
            vv = v[lo:a + i + 1].repeat_interleave(batch.group, 1)
            s = torch.einsum("hd,khd->hk", q[i], kk) * scale
            size = torch.einsum("hd,khd->hk", q[i].abs(), kk.abs()) * scale
            lse = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[:, None])
            o = torch.einsum("hk,khd->hd", p, vv)
            weight = torch.einsum("hk,khd->hd", p, vv.abs())
            keys = s.shape[1]
            ds = (size.amax(-1) * (D + 2) * 2.0 ** -24 + s.abs().amax(-1) * 2.0 ** -23 + 2.0 ** -20)[:, None]
            rel = u + 2 * ds + (keys + D) * 2.0 ** -23
            tols.append(u * o.abs() + weight * rel * (1 + u) + tiny * (1 + vv.abs().sum(0)))
            ltols.append(ds[:, 0] + keys * 2.0 ** -23 + 2.0 ** -22 * (1 + lse.abs()))
            outs.append(o)
            lses.append(lse)
    empty = torch.empty(0, batch.Hq, D, dtype=torch.float64)
    if not outs:
        return empty, empty[..., 0], empty, empty[..., 0]
    return torch.stack(outs), torch.stack(lses), torch.stack(tols), torch.stack(ltols)


def assert_within(got, want, tol, what):
    got = got.double().cpu()
    assert got.shape == want.shape
    bad = ~((got - want).abs() <= tol)
    if bool(bad.any()):
        at = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {at}: "
                             f"{float(got[at])} against {float(want[at])}, allowed {float(tol[at])}")


def rotation_table(positions, dim, base=10000.0):
    at = torch.arange(positions, dtype=torch.float64)[:, None]
    rate = base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    return torch.cat([(at * rate).cos(), (at * rate).sin()], 1).float()


def rotate64(x, table, interleaved):
    """(rotated, bound): x [n, heads, D] by the rows of table [n, dim], in 64 bits; two products and a sum
    in fp32, then one rounding (fp16's smallest results: half its smallest step)."""
    dim = table.shape[1]
    y, mag = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    for j in range(dim // 2):
        lo, hi = (2 * j, 2 * j + 1) if interleaved else (j, j + dim // 2)
        a, b = x[:, :, lo].double(), x[:, :, hi].double()
        c, s = table[:, None, j].double(), table[:, None, dim // 2 + j].double()
        y[:, :, lo], y[:, :, hi] = a * c - b * s, b * c + a * s
        mag[:, :, lo], mag[:, :, hi] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0
    return y, half_step(x.dtype) * y.abs() + mag * 2.0 ** -22 + tiny * (mag > 0)
