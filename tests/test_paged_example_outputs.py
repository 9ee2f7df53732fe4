"""The example's forwards: what every emitted token's chunk attended to is, within the roundings, what one pass over the
emitted text gives, and both are the formula's over what the caches hold."""
import os
import sys

import pytest
import torch

from paged_long import attention64_wide

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
def test_the_steps_attention_is_that_of_one_pass_over_the_text(monkeypatch):
    import paged_verify_step as ex
    import speculative_decoding_logit_gb300 as asv
    asv.build()
    calls = []
    attend = asv.paged_attention

    def record(q, k_cache, *rest, **kw):
        got = attend(q, k_cache, *rest, **kw)
        calls.append((k_cache.data_ptr(), q, rest[2].tolist(), rest[3].tolist(), got.out))
        return got

    monkeypatch.setattr(ex.asv, "paged_attention", record)
    full, short = ex.contexts_of(3, seed=5)
    steps = 6
    views, emitted, accepted = ex.decode(full, short, steps)
    for name, ctx in (("a", full), ("b", short), ("t", short)):
        view = views[name]
        text = [c + [x for x in emitted[r].flatten().tolist() if x >= 0] for r, c in enumerate(ctx)]
        lengths = [len(x) - 1 for x in text]
        again = ex.View(view.model, 3)
        before = len(calls)
        logits = again.forward(torch.tensor(sum((x[:-1] for x in text), []), device="cuda"), ex.packed(lengths))
        (_, q, _, starts, out), = calls[before:]
        assert torch.equal(logits, out.flatten(1) @ view.model.head)
        held = [[x[again.block_table[r].long()[at // ex.PAGE], at % ex.PAGE] for r, at in
                 enumerate(torch.arange(n, device="cuda") for n in lengths)] for x in (again.k_cache, again.v_cache)]
        b = type("Held", (), dict(q_lens=lengths, past=[0] * 3, k=held[0], v=held[1], qd=q, starts=starts, B=3, N=sum(lengths),
                                  dim=ex.DIM, group=ex.Q_HEADS // ex.KV_HEADS, Hkv=ex.KV_HEADS, dtype=torch.bfloat16))
        want = attention64_wide(b)
        for r, (o, _, tol, _) in want.items():
            assert bool(((out[starts[r]:starts[r + 1]].double() - o).abs() <= tol).all())
        rows = 0
        for ptr, _, cache_len, ptrs, got in calls[:before]:
            if ptr != view.k_cache.data_ptr() or [y - x for x, y in zip(ptrs, ptrs[1:])] != [3] * 3:
                continue
            for r in range(3):
                o, _, tol, _ = want[r]
                # the chunk's rows whose tokens were emitted
                at = cache_len[r] + torch.arange(3)
                keep = at < lengths[r]
                step = [c[2][r] for c in calls[:before] if c[0] == ptr and [y - x for x, y in zip(c[3], c[3][1:])] == [3] * 3]
                nxt = step[step.index(cache_len[r]) + 1] if step.index(cache_len[r]) + 1 < len(step) else lengths[r]
                keep &= at < nxt
                mine = got[ptrs[r]:ptrs[r + 1]][keep].double()
                assert bool(((mine - o[at[keep].cuda()]).abs() <= tol[at[keep].cuda()]).all())
                rows += int(keep.sum())
        assert rows == int((accepted + 1).sum())
