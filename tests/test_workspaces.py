"""Zero-filling the workspaces that calls without workspace= keep, which ASV_REQ_TIMEOUT asks for."""
import pytest
import torch

from paged_util import Batch


def test_kept_workspaces_are_zero_filled_in_place(monkeypatch):
    import speculative_decoding_logit_gb300 as asv
    from speculative_decoding_logit_gb300 import _binding
    verify, paged = torch.ones(5000, dtype=torch.uint8), torch.ones(9000, dtype=torch.uint8)
    waits = []
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: waits.append(bool(verify.any())))
    monkeypatch.setattr(_binding, "_ws_cache", {(0, 1): verify})
    monkeypatch.setattr(_binding, "_paged_ws_cache", {(0, 1): paged})
    asv.clear_workspaces()
    assert not verify.any() and not paged[:_binding.PAGED_WORKSPACE_ZEROED].any()
    assert waits[0] and not waits[-1]   # calls in flight end before, the fills before it returns
    assert _binding._ws_cache[0, 1] is verify and _binding._paged_ws_cache[0, 1] is paged   # (graphs may hold them)


@pytest.mark.gpu
def test_a_call_after_clearing_counts_from_zero():
    import speculative_decoding_logit_gb300 as asv
    from speculative_decoding_logit_gb300 import _binding
    asv.build()
    b = Batch([2, 9], [3000, 700], heads=(8, 2), dim=64, seed=3).fill()
    ref = asv.paged_attention(b.qd, b.k_cache, b.v_cache, b.table, b.cache_len, b.indptr)
    for ws in _binding._paged_ws_cache.values():
        ws[:_binding.PAGED_WORKSPACE_ZEROED] = 1   # as a call that gave up may leave them
    asv.clear_workspaces()
    got = asv.paged_attention(b.qd, b.k_cache, b.v_cache, b.table, b.cache_len, b.indptr)
    assert torch.equal(got.out, ref.out) and torch.equal(got.lse, ref.lse)
