"""Speculative decoding steps with the forwards' attention over paged caches and AsymSpec's verification.

  python examples/paged_verify_step.py [--steps N]

Three views of every request, as AsymSpec has them ("AsymSpec: Context-Asymmetric Speculative Decoding
for Agentic LLMs", sec. 4.1): the drafter on the full context (a), the drafter on the compressed
context (b), the verifier on the compressed context (t).  Each view has a paged key/value cache of its
own.  A step drafts K tokens one at a time on the full context, runs the chunk of K + 1 tokens through
the three views (append, attend, logits), verifies, and advances every view's cache_len by
accept_len + 1: the rejected drafts' slots are written over by the next step's append.  Lengths, tokens
and accept lengths stay on the GPU throughout.

The models are stand-ins of one attention layer with random weights: a token's query, key and value are
rows of a table, its logits the attention output times a matrix.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import speculative_decoding_logit_gb300 as asv  # noqa: E402

VOCAB, Q_HEADS, KV_HEADS, DIM, PAGE, MAX_LEN = 4096, 8, 2, 64, 16, 512


class Model:
    """One attention layer: token -> (q, k, v) by a table, attention output -> logits by a matrix."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)
        self.qkv = rand(VOCAB, (Q_HEADS + 2 * KV_HEADS) * DIM)
        self.head = rand(Q_HEADS * DIM, VOCAB) * (Q_HEADS * DIM) ** -0.5 * 4


class View:
    """A model over a batch's contexts, with a paged cache: requests' pages are handed out once."""

    def __init__(self, model, B):
        self.model = model
        pages = MAX_LEN // PAGE
        shape = (B * pages, PAGE, KV_HEADS, DIM)
        self.k_cache, self.v_cache = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        order = torch.randperm(B * pages, generator=torch.Generator().manual_seed(B))
        self.block_table = order.view(B, pages).to(torch.int32).cuda()
        self.cache_len = torch.zeros(B, dtype=torch.int32, device="cuda")
        at = torch.arange(MAX_LEN, dtype=torch.float64, device="cuda")[:, None]
        rate = 10000.0 ** (-torch.arange(0, DIM, 2, dtype=torch.float64, device="cuda") / DIM)
        self.rotary = torch.cat([(at * rate).cos(), (at * rate).sin()], 1).float()
        self.status = torch.zeros(B, dtype=torch.int32, device="cuda")

    def forward(self, tokens, indptr, cache_len=None):
        """Logits [N, VOCAB] of the packed chunks `tokens` behind what each request has in the cache."""
        cache_len = self.cache_len if cache_len is None else cache_len
        q, k, v = self.model.qkv[tokens.long()].split([Q_HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM], 1)
        q, k, v = (x.unflatten(1, (-1, DIM)) for x in (q, k, v))
        app = asv.paged_kv_append(k, v, self.k_cache, self.v_cache, self.block_table, cache_len, indptr, q=q,
                                  rotary=self.rotary)
        att = asv.paged_attention(app.q, self.k_cache, self.v_cache, self.block_table, cache_len, indptr)
        self.status |= app.req_status | att.req_status
        return att.out.flatten(1) @ self.model.head


def packed(lengths):
    return torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def decode(contexts, compressed, steps, K=2, beta=1.0, gamma=0.5):
    """Runs `steps` speculative steps; contexts and compressed are lists of token lists.  Returns the views,
    the emitted tokens [B, steps, K + 1] (-1 padded) and accept lengths [B, steps]."""
    B = len(contexts)
    drafter, verifier = Model(1), Model(2)
    verifier.qkv[:, :] = drafter.qkv + 0.1 * verifier.qkv    # alike, so that some drafts pass
    verifier.head[:, :] = drafter.head + 0.1 * verifier.head
    views = {"a": View(drafter, B), "b": View(drafter, B), "t": View(verifier, B)}
    # prompts: all but the last token of each context is written, the last opens the first chunk
    for name, ctx in (("a", contexts), ("b", compressed), ("t", compressed)):
        view, lengths = views[name], [len(c) - 1 for c in ctx]
        view.forward(torch.tensor(sum((c[:-1] for c in ctx), []), device="cuda"), packed(lengths))
        view.cache_len += torch.tensor(lengths, dtype=torch.int32, device="cuda")
    last = torch.tensor([c[-1] for c in contexts], dtype=torch.int32, device="cuda")
    one, chunk = packed([1] * B), packed([K + 1] * B)
    emitted, accepted = [], []
    for _ in range(steps):
        tokens = [last]
        for i in range(K):  # drafts, one token at a time on the full context
            logits = views["a"].forward(tokens[-1], one, views["a"].cache_len + i)
            tokens.append(logits.argmax(-1).to(torch.int32))
        rows = torch.stack(tokens, 1)
        a, b, t = (views[n].forward(rows.flatten(), chunk).view(B, K + 1, VOCAB) for n in "abt")
        out = asv.asymspec_verify(a, b, t, rows[:, 1:].contiguous(), beta, gamma)
        for view in views.values():
            view.cache_len += out.accept_len + 1
            view.status |= out.req_status
        last = out.tokens.gather(1, out.accept_len.long()[:, None])[:, 0]
        emitted.append(out.tokens)
        accepted.append(out.accept_len)
    return views, torch.stack(emitted, 1), torch.stack(accepted, 1)


def contexts_of(B, seed=0):
    g = torch.Generator().manual_seed(seed)
    full = [torch.randint(0, VOCAB, (int(n),), generator=g).tolist() for n in torch.randint(60, 300, (B,), generator=g)]
    return full, [c[::4] + c[-8:] for c in full]


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    args = ap.parse_args()
    asv.build()
    full, short = contexts_of(4)
    views, emitted, accepted = decode(full, short, args.steps)
    for r in range(len(full)):
        text = [int(x) for x in emitted[r].flatten().tolist() if x >= 0]
        print(f"request {r}: context {len(full[r])} ({len(short[r])} compressed), accepted per step "
              f"{accepted[r].tolist()}, tokens {text}")
    assert not any(bool(v.status.any()) for v in views.values())


if __name__ == "__main__":
    main()
