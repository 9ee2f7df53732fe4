"""sample_tokens of the bounds-checked library: its check log stays zero, canaries behind every output are intact, and the
results are the ordinary library's; two calls at once, and calls through graphs that run next to each other."""
import ctypes as C

import pytest
import torch

import test_paged_checked as small
import test_sample as sample

pytestmark = pytest.mark.gpu
libs = small.libs


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,n,V,kind", [(1, 1, 1, "peaked"), (2, 3, 17, "masked"), (1, 1, 1001, "flat"), (3, 2, 4099, "peaked"),
                                        (2, 1, 30001, "ties"), (1, 1, 151936, "flat"), (90, 1, 1003, "peaked"),
                                        (100, 2, 9001, "flat")])
def test_no_index_leaves_its_buffer(libs, dtype, B, n, V, kind):
    asv, m, lib = libs
    x, u = sample._logits_of(B, n, V, kind, dtype, V).cuda(), sample._draws(B, n, V).cuda()
    # the rows at the very end of what they lie in
    whole = torch.zeros(8 + x.numel(), dtype=dtype, device="cuda")
    whole[8 - V % 8:8 - V % 8 + x.numel()] = x.flatten()
    xs = whole[8 - V % 8:8 - V % 8 + x.numel()].view(B, n, V)
    i32 = dict(dtype=torch.int32, device="cuda")
    for T, k, p, least in ((1.0, 0, 1.0, 0.0), (0.9, 20, 0.9, 0.0), (1.0, 0, 0.9, 0.0), (0.0, 0, 1.0, 0.0), (1.2, 700, 0.99, 0.0),
                           (1.0, 0, 1.0, 0.05)):
        ref = asv.sample_tokens(xs, u, temperature=T, top_k=k, top_p=p, min_p=least, probs=True)
        g = {"tokens": torch.zeros(B, n, **i32), "logprobs": torch.zeros(B, n, device="cuda"),
             "probs": torch.zeros(B, n, V, device="cuda"), "status": torch.zeros(B, **i32)}
        g = {name: small.Guarded(t) for name, t in g.items()}
        field = lambda t: m._FieldC(t.data_ptr(), t.stride(0), t.stride(1))
        keep = [m._LogitsC(xs.data_ptr(), int(dtype == torch.bfloat16), B, n, V, xs.stride(0), xs.stride(1)), field(u),
                m._SamplingC(T, k, p, least), field(g["tokens"].t), field(g["logprobs"].t), field(g["probs"].t)]
        at = [C.addressof(s) for s in keep]
        assert lib.sample_tokens(at[0], at[1], at[2], None, at[3], at[4], at[5], g["status"].t.data_ptr(),
                                 torch.cuda.current_stream().cuda_stream) == 0
        log = (C.c_uint32 * 2)(9, 9)
        assert lib.asv_sample_check_log(log) == 0
        assert list(log) == [0, 0]
        assert all(s.intact() for s in g.values())
        assert torch.equal(g["tokens"].t, ref.tokens) and torch.equal(g["logprobs"].t, ref.logprobs)
        assert torch.equal(g["probs"].t, ref.probs) and not g["status"].t.any()


def _inputs(seed, B=200, V=6000):
    kind = "peaked" if seed % 2 else "flat"
    return sample._logits_of(B, 1, V, kind, torch.bfloat16, seed).cuda(), sample._draws(B, 1, seed).cuda()


def test_two_calls_at_once(libs):
    """Nothing is shared between calls: on two streams, many times, each gets what it gets alone."""
    asv = libs[0]
    calls = [_inputs(s) for s in range(2)]
    want = [asv.sample_tokens(x, u, top_p=0.9, probs=True) for x, u in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(asv.sample_tokens(*calls[i], top_p=0.9, probs=True, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert torch.equal(g.tokens, want[i].tokens) and torch.equal(g.probs, want[i].probs)
            assert torch.equal(g.logprobs, want[i].logprobs)


def test_two_graphs_at_once(libs):
    asv = libs[0]
    graphs, outs, want, streams = [], [], [], []
    for i in range(2):
        x, u = _inputs(10 + i)
        out = asv.sample_tokens(x, u, top_p=0.9, probs=True)
        want.append([t.clone() for t in (out.tokens, out.logprobs, out.probs)])
        for t in (out.tokens, out.logprobs, out.probs):
            t.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(5):
                asv.sample_tokens(x, u, top_p=0.9, out=out)
        graphs.append((g, x, u))
        outs.append(out)
        streams.append(torch.cuda.Stream())
    torch.cuda.synchronize()
    for _ in range(4):
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        for t, v in zip((out.tokens, out.logprobs, out.probs), w):
            assert torch.equal(t, v)
