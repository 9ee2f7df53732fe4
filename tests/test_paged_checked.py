"""The bounds-checked library's paged entry points through the C ABI, with canary words behind every
buffer they write (queries, outputs, log-sum-exps, caches, status, workspace): the check log stays
zero, every canary intact, the tickets zero, and the results are the ordinary library's."""
import ctypes as C

import pytest
import torch

from paged_util import Batch, rotation_table

pytestmark = pytest.mark.gpu
CANARY, GUARD = 0x5A, 512


@pytest.fixture(scope="module")
def libs():
    import speculative_decoding_logit_gb300 as asv
    from speculative_decoding_logit_gb300 import _binding, nvcc_build
    asv.build()
    lib = C.CDLL(nvcc_build.build_checked())
    _binding._declare(lib)
    return asv, _binding, lib


class Guarded:
    """A copy of `t` (strides kept) followed by GUARD canary bytes."""

    def __init__(self, t):
        self.n = (1 + sum((e - 1) * s for e, s in zip(t.shape, t.stride()))) * t.element_size()
        self.raw = torch.full((self.n + GUARD,), CANARY, dtype=torch.uint8, device="cuda")
        flat = self.raw[:self.n].view(t.dtype)
        self.t = torch.as_strided(flat, t.shape, t.stride())
        self.t.copy_(t)

    def intact(self):
        return bool((self.raw[self.n:] == CANARY).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q_lens,past,heads,dim,page,window,first", [
    ([1], [0], (1, 1), 8, 8, 0, False),
    ([3, 0, 40], [130, 5, 0], (6, 2), 40, 24, 0, False),
    ([1, 1, 1], [900, 17, 2600], (8, 2), 128, 16, 0, True),
    ([300, 1, 70], [10, 400, 129], (4, 1), 128, 64, 100, False),
    ([150, 139], [0, 700], (5, 5), 80, 48, 0, True),
])
def test_no_index_leaves_its_buffer(libs, dtype, q_lens, past, heads, dim, page, window, first):
    asv, m, lib = libs
    b = Batch(q_lens, past, heads=heads, dim=dim, page=page, dtype=dtype, heads_first=first, seed=len(q_lens)).fill(upto=past)
    table = rotation_table(max(a + n for a, n in zip(past, q_lens)), dim // 2 // 2 * 2).cuda()
    k, v = (x.cuda() for x in b.new_rows())
    ref_cache = b.k_cache.clone(), b.v_cache.clone()
    ref_q = asv.paged_kv_append(k, v, *ref_cache, b.table, b.cache_len, b.indptr, q=b.qd, rotary=table).q
    ref = asv.paged_attention(ref_q, *ref_cache, b.table, b.cache_len, b.indptr, window=window)

    kc, vc = Guarded(b.k_cache), Guarded(b.v_cache)
    q = Guarded(torch.zeros_like(b.qd))
    out, lse = Guarded(torch.zeros_like(ref.out)), Guarded(torch.zeros_like(ref.lse))
    status = Guarded(torch.zeros(b.B, dtype=torch.int32, device="cuda"))
    need = lib.asv_paged_workspace_bytes(heads[0], heads[1], dim)
    ws = Guarded(torch.zeros(need, dtype=torch.uint8, device="cuda"))
    assert ws.raw.data_ptr() % 256 == 0
    keep = [m._PagedCacheC(kc.t.data_ptr(), vc.t.data_ptr(), m.ASV_BF16 if dtype == torch.bfloat16 else m.ASV_F16,
                           *kc.t.shape, *kc.t.stride()[:3], *vc.t.stride()[:3]),
            m._PagedBatchC(b.B, b.N, b.indptr.data_ptr(), b.cache_len.data_ptr(), b.table.data_ptr(), b.table.shape[1],
                           b.table.stride(0)),
            m._RotaryC(table.data_ptr(), table.shape[1], table.shape[0], 0)]
    cache, batch, rot = (C.addressof(x) for x in keep)

    def rows(x):
        keep.append(m._RowsC(x.data_ptr(), x.stride(0), x.stride(1)))
        return C.addressof(keep[-1])
    sh = torch.cuda.current_stream().cuda_stream
    assert lib.paged_kv_append(cache, batch, rows(k), rows(v), rows(b.qd), rows(q.t), heads[0], rot,
                               status.t.data_ptr(), sh) == 0
    for _ in range(2):
        assert lib.paged_attention(cache, batch, rows(q.t), rows(out.t), heads[0], dim ** -0.5, window,
                                   lse.t.data_ptr(), status.t.data_ptr(), ws.t.data_ptr(), need, sh) == 0
    torch.cuda.synchronize()
    for g in (kc, vc, q, out, lse, status, ws):
        assert g.intact()
    assert not status.t.any()
    assert not ws.t[:4096].any()                       # tickets
    assert not ws.t[need - 256:].any()                 # check log
    nan = lambda x: torch.nan_to_num(x.float(), nan=-7.0)
    assert torch.equal(q.t, ref_q) and torch.equal(out.t, ref.out) and torch.equal(lse.t, ref.lse)
    assert torch.equal(nan(kc.t), nan(ref_cache[0])) and torch.equal(nan(vc.t), nan(ref_cache[1]))
