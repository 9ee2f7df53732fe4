"""paged_kv_append of the bounds-checked library: its check log (kept by the library, as the append has no workspace) stays
zero over rotations, tokens to a CTA, and batches with bad pages and lengths; every canary behind what it writes is intact;
and the results are the ordinary library's."""
import ctypes as C

import pytest
import torch

import test_paged_checked as small
from paged_util import Batch, rotation_table

pytestmark = pytest.mark.gpu
libs = small.libs


def _many(n):
    q = [1, 0, 7, 2, 31, 3, 0, 0, 5, 1]
    return q + [n - sum(q) - 40, 37, 3]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q_lens,heads,dim,page,rot,interleaved,bad", [
    ([3, 1, 40], (6, 2), 64, 16, 64, False, False),    # whole halves
    ([3, 1, 40], (6, 2), 64, 24, 40, False, True),     # partners by four
    ([3, 1, 40], (5, 5), 120, 8, 90, False, False),    # partners one by one
    ([3, 0, 40], (28, 4), 128, 64, 64, True, True),    # neighbours
    ([9, 2, 5], (2, 1), 8, 16, 0, False, False),       # no rotation
    (_many(2500), (1, 1), 16, 16, 8, False, False),    # two to sixteen tokens to a CTA
    (_many(5000), (1, 1), 16, 16, 16, False, True),
    (_many(10000), (1, 1), 16, 16, 2, False, False),
])
def test_no_index_of_an_append_leaves_its_buffer(libs, dtype, q_lens, heads, dim, page, rot, interleaved, bad):
    asv, m, lib = libs
    past = [(53 * i) % 90 for i in range(len(q_lens))]
    b = Batch(q_lens, past, heads=heads, dim=dim, page=page, dtype=dtype, seed=dim).fill(upto=past)
    if bad:
        b.cache_len[0] = -5
        b.table[1:, 0] = -7
        b.table[2, 1] = 1 << 30
        b.cache_len[-1] = b.table.shape[1] * page
    k, v = (x.cuda() for x in b.new_rows())
    table = rotation_table(max(a + n for a, n in zip(past, q_lens)), rot).cuda() if rot else None
    ref_cache = b.k_cache.clone(), b.v_cache.clone()
    ref_out = asv.PagedAppendOutput(torch.zeros_like(b.qd), torch.zeros(b.B, dtype=torch.int32, device="cuda"))
    ref = asv.paged_kv_append(k, v, *ref_cache, b.table, b.cache_len, b.indptr, q=b.qd, rotary=table,
                              interleaved=interleaved, out=ref_out)
    kc, vc, q = small.Guarded(b.k_cache), small.Guarded(b.v_cache), small.Guarded(torch.zeros_like(b.qd))
    status = small.Guarded(torch.zeros(b.B, dtype=torch.int32, device="cuda"))
    keep = [m._PagedCacheC(kc.t.data_ptr(), vc.t.data_ptr(), m.ASV_BF16 if dtype == torch.bfloat16 else m.ASV_F16,
                           *kc.t.shape, *kc.t.stride()[:3], *vc.t.stride()[:3]),
            m._PagedBatchC(b.B, b.N, b.indptr.data_ptr(), b.cache_len.data_ptr(), b.table.data_ptr(), b.table.shape[1],
                           b.table.stride(0)),
            m._RotaryC(table.data_ptr(), rot, table.shape[0], int(interleaved)) if rot else None]
    cache, batch, rotary = (None if x is None else C.addressof(x) for x in keep)

    def rows(x):
        keep.append(m._RowsC(x.data_ptr(), x.stride(0), x.stride(1)))
        return C.addressof(keep[-1])
    assert lib.paged_kv_append(cache, batch, rows(k), rows(v), rows(b.qd), rows(q.t), heads[0], rotary, status.t.data_ptr(),
                               torch.cuda.current_stream().cuda_stream) == 0
    log = (C.c_uint32 * 2)(9, 9)
    assert lib.asv_paged_append_check_log(log) == 0
    assert list(log) == [0, 0]
    for g in (kc, vc, q, status):
        assert g.intact()
    assert status.t.tolist() == ref.req_status.tolist() and bool(status.t.any()) == bad
    nan = lambda x: torch.nan_to_num(x.float(), nan=-7.0)
    assert torch.equal(q.t, ref.q)
    assert torch.equal(nan(kc.t), nan(ref_cache[0])) and torch.equal(nan(vc.t), nan(ref_cache[1]))
