"""Refusals of the paged-cache entry points, on the host: each case leaves every pointer NULL except
the one it checks, so a regression in a check ends at ASV_ERR_NULL and no case can reach a launch."""
import ctypes as C

import pytest
import torch

NULL, SHAPE, ALIGN, DTYPE, PARAM = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def m():
    import speculative_decoding_logit_gb300 as asv
    asv.build()
    asv.library()
    from speculative_decoding_logit_gb300 import _binding
    return _binding


host = (C.c_uint64 * 64)()  # a real allocation: misaligned addresses are taken inside it
BASE = (C.addressof(host) + 255) // 256 * 256


def _cache(m, **kw):
    c = dict(k=None, v=None, dtype=1, num_pages=4, page_size=16, kv_heads=2, head_dim=64, k_stride_page=2048,
             k_stride_slot=128, k_stride_head=64, v_stride_page=2048, v_stride_slot=128, v_stride_head=64)
    c.update(kw)
    return m._PagedCacheC(**c)


def _batch(m, **kw):
    b = dict(B=2, N=3, indptr=None, cache_len=None, block_table=None, max_pages=2, block_table_stride=2)
    b.update(kw)
    return m._PagedBatchC(**b)


def _append(m, cache=None, batch=None, k=None, v=None, q=None, oq=None, heads=4, rot=None):
    ref = lambda x: None if x is None else C.addressof(x)
    cache, batch = cache or _cache(m), batch or _batch(m)
    return m.library().paged_kv_append(C.addressof(cache), C.addressof(batch), ref(k), ref(v), ref(q), ref(oq), heads,
                                       ref(rot), None, None)


def _attend(m, cache=None, batch=None, q=None, out=None, heads=4, scale=0.125, window=0, lse=None, ws=None, n=0):
    ref = lambda x: None if x is None else C.addressof(x)
    cache, batch = cache or _cache(m), batch or _batch(m)
    return m.library().paged_attention(C.addressof(cache), C.addressof(batch), ref(q), ref(out), heads, scale, window,
                                       lse, None, ws, n, None)


SIZES = [("page_size", 0), ("page_size", 4), ("page_size", 12), ("kv_heads", 0), ("kv_heads", 2000), ("head_dim", 0),
         ("head_dim", 60), ("head_dim", 136), ("num_pages", -1)]


@pytest.mark.parametrize("field,value", SIZES)
@pytest.mark.parametrize("call", [_append, _attend])
def test_cache_sizes(m, call, field, value):
    assert call(m, cache=_cache(m, **{field: value})) == SHAPE


@pytest.mark.parametrize("field,value", [("B", -1), ("N", -1), ("max_pages", -1), ("max_pages", 1 << 28)])
@pytest.mark.parametrize("call", [_append, _attend])
def test_batch_sizes(m, call, field, value):
    assert call(m, batch=_batch(m, **{field: value})) == SHAPE


@pytest.mark.parametrize("call", [_append, _attend])
def test_element_types(m, call):
    assert call(m, cache=_cache(m, dtype=0)) == DTYPE   # fp32 logits are no cache type
    assert call(m, cache=_cache(m, dtype=7)) == DTYPE
    assert call(m, cache=_cache(m, dtype=2)) == NULL


@pytest.mark.parametrize("call", [_append, _attend])
def test_empty_batches_are_no_ops(m, call):
    assert call(m, batch=_batch(m, B=0)) == 0
    assert call(m, batch=_batch(m, N=0)) == 0


@pytest.mark.parametrize("call", [_append, _attend])
@pytest.mark.parametrize("field,value", [("k", BASE + 8), ("v", BASE + 2), ("k_stride_slot", 132), ("v_stride_head", 0),
                                         ("k_stride_page", -2048), ("v_stride_page", 4)])
def test_cache_alignment(m, call, field, value):
    assert call(m, cache=_cache(m, **{field: value})) == ALIGN


@pytest.mark.parametrize("call", [_append, _attend])
@pytest.mark.parametrize("field", ["indptr", "cache_len", "block_table"])
def test_batch_alignment(m, call, field):
    assert call(m, batch=_batch(m, **{field: BASE + 2})) == ALIGN


def test_strides_of_single_entries_are_not_looked_at(m):
    c = _cache(m, num_pages=1, kv_heads=1, k_stride_page=3, v_stride_page=0, k_stride_head=-5, v_stride_head=1)
    assert _append(m, cache=c) == NULL
    assert _attend(m, cache=c) == NULL


@pytest.mark.parametrize("data,tok,head", [(BASE + 8, 256, 64), (BASE, 0, 64), (BASE, 256, 60), (BASE, -256, 64)])
def test_row_alignment(m, data, tok, head):
    r = m._RowsC(data, tok, head)
    for name in ("k", "v", "q", "oq"):
        assert _append(m, **{name: r}) == ALIGN
    for name in ("q", "out"):
        assert _attend(m, **{name: r}) == ALIGN


@pytest.mark.parametrize("kw", [dict(dim=0), dict(dim=7), dict(dim=66), dict(max_position=0), dict(interleaved=2)])
def test_rotation_sizes(m, kw):
    r = dict(table=None, dim=64, max_position=10, interleaved=0)
    r.update(kw)
    assert _append(m, rot=m._RotaryC(**r)) == PARAM


def test_rotation_alignment(m):
    assert _append(m, rot=m._RotaryC(BASE + 2, 64, 10, 0)) == ALIGN


@pytest.mark.parametrize("heads", [0, -2, 3, 2 * 129])
def test_query_heads(m, heads):
    assert _attend(m, heads=heads) == SHAPE


def test_attention_scalars(m):
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _attend(m, scale=scale) == PARAM
    assert _attend(m, window=-1) == PARAM
    assert _attend(m, lse=BASE + 2) == ALIGN
    assert _attend(m, ws=BASE + 16) == ALIGN
    assert _attend(m) == NULL
    assert m.library().paged_attention(None, None, None, None, 4, 1.0, 0, None, None, None, 0, None) == NULL
    assert m.library().paged_kv_append(None, None, None, None, None, None, 4, None, None, None) == NULL


def test_workspace_size(m):
    n = m.paged_workspace_bytes(32, 8, 128)
    assert n > 0
    for bad in ((32, 0, 128), (2, 4, 128), (4, 4, 0)):
        assert m.paged_workspace_bytes(*bad) == 0


def test_binding_refuses_host_tensors():
    import speculative_decoding_logit_gb300 as asv
    c = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(asv.AsvError):
        asv.paged_attention(torch.zeros(1, 4, 64, dtype=torch.bfloat16), c, c, i[None], i, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(asv.AsvError):
        asv.paged_kv_append(c[0, :1], c[0, :1], c, c, i[None], i, torch.zeros(2, dtype=torch.int32))


@pytest.mark.gpu
def test_binding_refuses_shapes_and_types():
    import speculative_decoding_logit_gb300 as asv
    asv.build()
    bf = dict(dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    c, q = torch.zeros(2, 16, 2, 64, **bf), torch.zeros(1, 4, 64, **bf)
    t, n, p = torch.zeros(1, 1, **i32), torch.zeros(1, **i32), torch.tensor([0, 1], **i32)
    ok = dict(q=q, k_cache=c, v_cache=c, block_table=t, cache_len=n, indptr=p)
    asv.paged_attention(**ok)

    def status(**kw):
        with pytest.raises(asv.AsvError) as e:
            asv.paged_attention(**{**ok, **kw})
        return e.value.status

    assert status(q=q.half()) == DTYPE
    assert status(q=q[0]) == SHAPE
    assert status(q=q[:, :3]) == SHAPE                       # 3 query heads to 2 key heads
    assert status(q=torch.zeros(1, 4, 32, **bf)) == SHAPE
    assert status(q=q.expand(3, 4, 64)) == ALIGN             # a stride of 0
    assert status(k_cache=c.float(), v_cache=c.float()) == DTYPE
    assert status(v_cache=c[:1]) == SHAPE
    assert status(cache_len=n.long()) == DTYPE
    assert status(indptr=p[:1]) == SHAPE
    assert status(block_table=t[0]) == SHAPE
    assert status(scale=-1.0) == PARAM
    assert status(window=-3) == PARAM
    assert status(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")) == 6
    k = c[0, :1]
    with pytest.raises(asv.AsvError):
        asv.paged_kv_append(k, k, c, c, t, n, p, rotary=torch.zeros(4, 66, device="cuda"))
    with pytest.raises(asv.AsvError):
        asv.paged_kv_append(k, k, c, c, t, n, p, rotary=torch.zeros(4, 64, device="cuda", dtype=torch.float64))
    with pytest.raises(asv.AsvError):
        asv.paged_kv_append(k.half(), k, c, c, t, n, p)
