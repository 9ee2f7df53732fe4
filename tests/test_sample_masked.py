"""Vocabularies of which long stretches are masked, as a constrained decoder and a padded vocabulary have them: whole CTAs' runs
without a token."""
import ctypes as C
import math

import pytest
import torch

import test_paged_checked as small
import test_paged_refusals as host
import test_sample as sample

m = host.m
libs = small.libs
BF, F32 = torch.bfloat16, torch.float32
PARAMETERS = ((1.0, 0, 1.0, 0.0), (0.9, 40, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (0.8, 300, 0.95, 0.01), (1.3, 0, 0.9, 0.05),
              (0.0, 0, 1.0, 0.0), (1.0, 3000, 0.9, 0.0), (1.0, 0, 1.0, 0.02))


def _masked(B, V, stretch, value, dtype):
    x = sample._logits_of(B, 1, V, "peaked", dtype, V + B)
    value = -math.inf if value == "none" else torch.finfo(dtype).min
    keep = torch.zeros(V, dtype=torch.bool)
    if stretch == "first":           # all but the first tenth
        keep[:V // 10] = True
    elif stretch == "padded":        # the last third
        keep[:V - V // 3] = True
    elif stretch == "behind":        # all but the last 50
        keep[-50:] = True
    elif stretch == "middle":
        keep[V // 2:V // 2 + 1000] = True
    elif stretch == "one":
        keep[V // 3] = True
    elif stretch == "few":           # 40 tokens allowed, anywhere
        keep[torch.randperm(V, generator=torch.Generator().manual_seed(V))[:40]] = True
    x[:, :, ~keep] = value
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B", [2, 90])
@pytest.mark.parametrize("value", ["none", "lowest"])
@pytest.mark.parametrize("stretch", ["first", "padded", "behind", "middle", "one", "few"])
def test_masked_stretches(m, dtype, B, value, stretch):
    V = 20011
    x, u = _masked(B, V, stretch, value, dtype), sample._draws(B, 1, B)
    few = slice(0, B, 1 + B // 8)
    for T, k, p, least in PARAMETERS:
        got = m.sample_tokens(x.cuda(), u.cuda(), temperature=T, top_k=k, top_p=p, min_p=least, probs=True)
        got = m.SampleOutput(*(t.cpu()[few] for t in (got.tokens, got.logprobs, got.probs, got.req_status)))
        sample._compare(x[few], u[few], got, T, k, p, least)


@pytest.mark.gpu
@pytest.mark.parametrize("ctas", range(1, 9))
@pytest.mark.parametrize("B", [1, 80])
def test_what_is_chosen_by_are_numbers(libs, ctas, B):
    """The checked library's log stays zero, at any number of CTAs, with whole runs masked."""
    asv, b, lib = libs
    V = 30011
    i32 = dict(dtype=torch.int32, device="cuda")
    assert lib.asv_set_tuning(ctas, 0) == 0
    try:
        for dtype in (BF, F32):
            for stretch in ("first", "padded", "behind", "few"):
                x, u = _masked(B, V, stretch, "none", dtype).cuda(), sample._draws(B, 1, B).cuda()
                for T, k, p, least in PARAMETERS:
                    want = asv.sample_tokens(x, u, temperature=T, top_k=k, top_p=p, min_p=least)
                    tokens, logs, status = torch.zeros(B, 1, **i32), torch.zeros(B, 1, device="cuda"), torch.zeros(B, **i32)
                    field = lambda t: b._FieldC(t.data_ptr(), t.stride(0), t.stride(1))
                    keep = [b._LogitsC(x.data_ptr(), int(dtype == BF), B, 1, V, V, V), field(u), b._SamplingC(T, k, p, least),
                            field(tokens), field(logs)]
                    at = [C.addressof(s) for s in keep]
                    assert lib.sample_tokens(at[0], at[1], at[2], None, at[3], at[4], None, status.data_ptr(),
                                             torch.cuda.current_stream().cuda_stream) == 0
                    log = (C.c_uint32 * 2)(9, 9)
                    assert lib.asv_sample_check_log(log) == 0
                    assert list(log) == [0, 0], (dtype, stretch, T, k, p, least)
                    assert torch.equal(tokens, want.tokens) and not status.any()
    finally:
        lib.asv_set_tuning(0, 0)
