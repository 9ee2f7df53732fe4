"""The example's speculative steps over paged caches: what the caches hold at the end is, bit for bit,
what the emitted text written in one chunk gives, and the forward over it gives the same logits."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
def test_steps_leave_the_caches_as_one_pass_over_the_text_does():
    import paged_verify_step as ex
    import speculative_decoding_logit_gb300 as asv
    asv.build()
    full, short = ex.contexts_of(3, seed=5)
    steps = 6
    views, emitted, accepted = ex.decode(full, short, steps)
    assert not any(bool(v.status.any()) for v in views.values())
    assert tuple(accepted.shape) == (3, steps) and bool(((accepted >= 0) & (accepted <= 2)).all())
    for name, ctx in (("a", full), ("t", short)):
        text = [c + [x for x in emitted[r].flatten().tolist() if x >= 0] for r, c in enumerate(ctx)]
        view = views[name]
        # the last emitted token is not in the caches yet
        assert view.cache_len.tolist() == [len(x) - 1 for x in text]
        again = ex.View(view.model, 3)
        lengths = [len(x) - 1 for x in text]
        again.forward(torch.tensor(sum((x[:-1] for x in text), []), device="cuda"), ex.packed(lengths))
        for r, n in enumerate(lengths):
            at = torch.arange(n, device="cuda")
            for old, new in ((view.k_cache, again.k_cache), (view.v_cache, again.v_cache)):
                x = old[view.block_table[r].long()[at // ex.PAGE], at % ex.PAGE]
                y = new[again.block_table[r].long()[at // ex.PAGE], at % ex.PAGE]
                assert torch.equal(x, y)
