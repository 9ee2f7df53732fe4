"""Cases, plain forms and 64-bit values of the two operators over a paged key/value cache:

- ``paged_kv_append``: the new tokens' keys and values into the cache's pages, keys (and queries)
  turned by their positions on the way;
- ``paged_attention``: the chunk of new tokens of every request attending over that cache, causal,
  grouped heads, with an optional sliding window.

Requests are packed: request b has the rows indptr[b] .. indptr[b + 1] of q, k and v, and
cache_len[b] tokens in the cache before them.  A chunk is what one forward of a model sees: one token
(plain decoding), K drafts and one more (the forward whose logits the verification takes), a piece of
a prompt, or all of it.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One request, one new token over a few thousand: the latency of a decoding step.
        _attend("attend_decode_b1", B=1, q=(1, 1), past=(4095, 4095), heads=(32, 8), dim=128, page=16),
        # K = 2 drafts on a compressed context, half precision, three query heads to a shared one.
        _attend("attend_verify_b4_short", B=4, q=(3, 3), past=(480, 620), heads=(24, 8), dim=64, page=32, type="f16"),
        # The verification batch of 64 requests, K = 2, contexts from 500 tokens to 12 thousand.
        _attend("attend_verify_b64_k2", B=64, q=(3, 3), past=(500, 12000), heads=(64, 8), dim=128, page=16),
        # Ten drafts and one over the full long context, a handful of requests.
        _attend("attend_verify_b4_g10_long", B=4, q=(11, 11), past=(110000, 124000), heads=(32, 8), dim=128, page=64),
        # Plain decoding of 256 ragged requests, pages with the heads outside.
        _attend("attend_decode_b256", B=256, q=(1, 1), past=(1, 4096), heads=(32, 8), dim=128, page=16, type="f16",
                heads_first=True),
        # Chunks of prompts over what is there already: arithmetic bound.
        _attend("attend_chunk_b4_2048", B=4, q=(2048, 2048), past=(6144, 6144), heads=(32, 8), dim=128, page=64),
        # Whole prompts of different lengths, nothing in the cache before.
        _attend("attend_prompt_b6_ragged", B=6, q=(333, 4096), past=(0, 0), heads=(32, 4), dim=128, page=128),
        # Chunks, drafts and single tokens in one batch under a sliding window; an odd head size and
        # page size, one key head to each query head.
        _attend("attend_mixed_window", B=8, q=(0, 700), past=(0, 3300), heads=(12, 12), dim=80, page=24, window=1024),
        # One token appended: the latency of the call.
        _append("append_decode_b1", B=1, q=(1, 1), past=(4095, 4095), heads=(32, 8), dim=128, page=16),
        # The same verification batch of 64 requests, K = 2.
        _append("append_verify_b64_k2", B=64, q=(3, 3), past=(500, 12000), heads=(64, 8), dim=128, page=16),
        # The batch of 1024 requests, K = 8; interleaved pairs, part of each head turned.
        _append("append_verify_b1024_k8", B=1024, q=(9, 9), past=(1, 1000), heads=(28, 4), dim=128, page=32,
                rotary=64, interleaved=True, type="f16"),
        # Long prompts written for the first time.
        _append("append_prompt_b8_ragged", B=8, q=(1000, 8192), past=(0, 0), heads=(32, 8), dim=128, page=64),
    ]


def _attend(name, *, B, q, past, heads, dim, page, type="bf16", window=0, heads_first=False, lens=1):
    return {"name": name, "op": "attend", "B": B, "q_lo": q[0], "q_hi": q[1], "past_lo": past[0], "past_hi": past[1],
            "q_heads": heads[0], "kv_heads": heads[1], "dim": dim, "page": page, "type": type, "window": window,
            "heads_first": heads_first, "lens": lens}


def _append(name, *, B, q, past, heads, dim, page, type="bf16", rotary=None, interleaved=False, heads_first=False,
            lens=1):
    return {"name": name, "op": "append", "B": B, "q_lo": q[0], "q_hi": q[1], "past_lo": past[0], "past_hi": past[1],
            "q_heads": heads[0], "kv_heads": heads[1], "dim": dim, "page": page, "type": type,
            "rotary": dim if rotary is None else rotary, "interleaved": interleaved, "heads_first": heads_first,
            "lens": lens}


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    while True:
        common = dict(page=rng.choice([8, 16, 24, 32, 48, 64, 128, 256]), type=rng.choice(["bf16", "f16"]),
                      heads_first=rng.random() < 0.3, lens=rng.randrange(1 << 30))
        kv_heads = rng.choice([1, 2, 4, 5, 8, 12])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        dim = rng.choice([64, 128, 128, 128, 80, 96, 40, 120])
        if kv_heads * group > 64:
            continue
        kind = rng.choice(["decode", "verify", "chunk", "prompt", "mixed"])
        if kind == "decode":
            B, q_lo, q_hi, past_hi = _log_int(rng, 1, 300), 1, 1, _log_int(rng, 64, 60000)
            past_lo = rng.choice([1, past_hi // 3 + 1, past_hi])
        elif kind == "verify":
            B, q_lo, past_hi = _log_int(rng, 1, 128), rng.choice([2, 3, 5, 9, 11, 17]), _log_int(rng, 64, 120000)
            q_hi, past_lo = q_lo, rng.choice([1, past_hi // 3 + 1, past_hi])
        elif kind == "chunk":
            B, q_hi, past_hi = _log_int(rng, 1, 8), _log_int(rng, 64, 2500), _log_int(rng, 64, 16000)
            q_lo, past_lo = rng.choice([q_hi, q_hi // 2 + 1]), past_hi // 2 + 1
        elif kind == "prompt":
            B, q_hi, past_hi, past_lo = _log_int(rng, 1, 8), _log_int(rng, 16, 6000), 0, 0
            q_lo = rng.choice([q_hi, q_hi // 4 + 1, 1])
        else:
            B, q_lo, q_hi = _log_int(rng, 2, 12), rng.choice([0, 1]), _log_int(rng, 16, 800)
            past_lo, past_hi = 0, _log_int(rng, 64, 4000)
        args = dict(B=B, q=(q_lo, q_hi), past=(past_lo, past_hi), heads=(kv_heads * group, kv_heads), dim=dim, **common)
        if rng.random() < 0.3:
            case = _append("", rotary=rng.choice([dim, dim, max(2, dim // 4 // 2 * 2)]),
                           interleaved=rng.random() < 0.4, **args)
        else:
            case = _attend("", window=rng.choice([0, 0, 0, _log_int(rng, 16, 4000)]), **args)
        del case["name"]
        ql, past = _lengths(case)
        total = [a + b for a, b in zip(ql, past)]
        cache = 4 * kv_heads * dim * sum(total)
        if not sum(ql) or B * max(total) > 3e5 * common["page"]:
            continue
        if case["op"] == "append":
            if sum(ql) * dim * kv_heads * (group + 2) > 1.4e8 or cache > 1.9e9:
                continue
        elif B * max(ql) * max(total) * kv_heads * group > 2.1e9 or cache > 1.9e9 \
                or B * max(total) * kv_heads * dim > 5e8 or work(case)["flops"] > 9e11:
            continue
        if 3 * 1024 in (kv_heads * dim, kv_heads * group * dim, kv_heads * (group + 2) * dim, max(ql), max(total)):
            continue
        return case


def _lengths(case):
    """New tokens and tokens in the cache before them, per request."""
    rng = random.Random(case["lens"])

    def spread(lo, hi):
        if lo == hi:
            return lo
        return int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1)))) - 1 if lo == 0 else _log_int(rng, lo, hi)

    B = case["B"]
    return [spread(case["q_lo"], case["q_hi"]) for _ in range(B)], \
        [spread(case["past_lo"], case["past_hi"]) for _ in range(B)]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev, dt = "cuda", _TYPES[case["type"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    ql, past = _lengths(case)
    B, Hq, Hkv, D, page = case["B"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    N = sum(ql)
    pages = [-(-(a + b) // page) for a, b in zip(ql, past)]
    width = max(pages)
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table, at = [], 0
    for n in pages:
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    starts = [0]
    for n in ql:
        starts.append(starts[-1] + n)

    def rand(*shape, gain=1.0):
        return torch.randn(*shape, dtype=dt, device=dev, generator=g) * gain

    def cache():
        # every slot holds something: what is past a request's tokens is some other request's past
        if case["heads_first"]:
            return rand(n_pages, Hkv, page, D).transpose(1, 2)
        return rand(n_pages, page, Hkv, D)

    i32 = dict(dtype=torch.int32, device=dev)
    s = {"op": case["op"], "k_cache": cache(), "v_cache": cache(), "block_table": torch.tensor(table, **i32),
         "cache_len": torch.tensor(past, **i32), "indptr": torch.tensor(starts, **i32), "q_max": max(ql),
         "kv_max": max(a + b for a, b in zip(ql, past)), "status": torch.zeros(B, **i32)}
    if case["op"] == "attend":
        s |= {"q": rand(N, Hq, D, gain=2.0), "scale": D ** -0.5, "window": case["window"],
              "out": torch.empty(N, Hq, D, dtype=dt, device=dev),
              "lse": torch.empty(N, Hq, dtype=torch.float32, device=dev)}
    else:
        # q, k and v are views of one projection's output, as a model makes them
        qkv = rand(N, (Hq + 2 * Hkv) * D)
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1))
        R = case["rotary"]
        at = torch.arange(s["kv_max"], dtype=torch.float64, device=dev)[:, None]
        rate = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=dev) / R)
        s |= {"q": q, "k": k, "v": v, "rotary": torch.cat([(at * rate).cos(), (at * rate).sin()], 1).float(),
              "interleaved": case["interleaved"], "q_out": torch.empty(N, Hq, D, dtype=dt, device=dev)}
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        import speculative_decoding_logit_gb300 as asv
        if s["op"] == "attend":
            out = asv.PagedAttentionOutput(s["out"], s["lse"], s["status"])
            asv.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cache_len"], s["indptr"],
                                scale=s["scale"], window=s["window"], out=out)
            return {"out": out.out, "lse": out.lse}
        out = asv.PagedAppendOutput(s["q_out"], s["status"])
        asv.paged_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["cache_len"], s["indptr"],
                            q=s["q"], rotary=s["rotary"], interleaved=s["interleaved"], out=out)
        return {"q": out.q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return _attend_plain(s) if s["op"] == "attend" else _append_plain(s)


def _rows(s, n):
    """Request and place in its chunk of every packed row."""
    row = torch.arange(n, device="cuda")
    request = torch.searchsorted(s["indptr"][1:].long(), row, right=True)
    return request, row - s["indptr"].long()[request]


def _attend_plain(s):
    q, table, start = s["q"], s["block_table"].long(), s["indptr"].long()
    N, Hq, D = q.shape
    B, Hkv, page = table.shape[0], s["k_cache"].shape[2], s["k_cache"].shape[1]
    past, count = s["cache_len"].long(), start[1:] - start[:-1]
    place = torch.arange(s["q_max"], device="cuda")
    chunk = q[(start[:-1, None] + place).clamp(max=N - 1)].float()          # [B, q_max, Hq, D]
    chunk = chunk.reshape(B, s["q_max"], Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    used = table[:, :-(-s["kv_max"] // page)].clamp(min=0)
    k = s["k_cache"][used].flatten(1, 2)[:, :s["kv_max"]].float().permute(0, 2, 3, 1)   # [B, Hkv, D, kv_max]
    v = s["v_cache"][used].flatten(1, 2)[:, :s["kv_max"]].float().transpose(1, 2)       # [B, Hkv, kv_max, D]
    score = ((chunk @ k) * s["scale"]).reshape(B, Hkv, -1, s["q_max"], s["kv_max"])
    at, key = (past[:, None] + place)[:, :, None], torch.arange(s["kv_max"], device="cuda")
    seen = (key <= at) & (key < (past + count)[:, None, None])
    if s["window"]:
        seen &= key > at - s["window"]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    weight = score.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    out = (weight.reshape(B, Hkv, -1, s["kv_max"]) @ v).reshape(B, Hkv, -1, s["q_max"], D) / total
    lse = (top + total.log()).squeeze(-1)
    request, i = _rows(s, N)
    return {"out": out[request, :, :, i].reshape(N, Hq, D).to(q.dtype), "lse": lse[request, :, :, i].reshape(N, Hq)}


def _append_plain(s):
    request, i = _rows(s, s["k"].shape[0])
    at = s["cache_len"].long()[request] + i
    page = s["k_cache"].shape[1]
    to = s["block_table"].long()[request, at // page], at % page
    s["k_cache"][to] = _turn_plain(s["k"], s["rotary"][at], s["interleaved"])
    s["v_cache"][to] = s["v"]
    return {"q": _turn_plain(s["q"], s["rotary"][at], s["interleaved"]), "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


def _turn_plain(x, table, interleaved):
    R = table.shape[1]
    cos, sin = table[:, None, :R // 2], table[:, None, R // 2:]
    y, turned = x.float(), x[..., :R].float()
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :R // 2], turned[..., R // 2:])
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)
    return torch.cat([turned, y[..., R:]], -1).to(x.dtype)


# ------------------------------------------------------------------ floors and 64-bit values

def work(case):
    ql, past = _lengths(case)
    Hq, Hkv, D, N = case["q_heads"], case["kv_heads"], case["dim"], sum(ql)
    if case["op"] == "append":
        table_rows = len({a + i for a, n in zip(past, ql) for i in range(n)})
        moved = 2 * 2 * N * (Hq + 2 * Hkv) * D + 4 * table_rows * case["rotary"]
        return {"bytes": moved + 4 * (2 * case["B"] + N), "flops": 3 * N * (Hq + Hkv) * case["rotary"]}
    pairs = keys = 0
    for n, a in zip(ql, past):
        if not n:
            continue
        w = case["window"] or a + n
        # token i sees min(a + i + 1, w) keys
        full = max(0, min(n, w - a))
        pairs += full * a + full * (full + 1) // 2 + (n - full) * w
        keys += a + n - max(0, a + 1 - w)
    moved = 2 * 2 * N * Hq * D + 4 * N * Hq + 2 * 2 * keys * Hkv * D
    return {"bytes": moved + 4 * (2 * case["B"] + -(-keys // case["page"])), "flops": 4 * pairs * Hq * D}


def exact(case, seed):
    s = prepare(case, seed)
    ql, past = _lengths(case)
    page, first = case["page"], 0
    if case["op"] == "append":
        kc, vc, q_new = s["k_cache"].double(), s["v_cache"].double(), s["q"].double()
        half = case["rotary"] // 2
        lo = [2 * j for j in range(half)] if case["interleaved"] else list(range(half))
        hi = [2 * j + 1 for j in range(half)] if case["interleaved"] else list(range(half, 2 * half))
        k_new = s["k"].double()
        for n, a in zip(ql, past):
            rows = slice(first, first + n)
            cos = s["rotary"][a:a + n, None, :half].double()
            sin = s["rotary"][a:a + n, None, half:].double()
            for x in (q_new, k_new):
                u, w = x[rows][..., lo], x[rows][..., hi]
                x[rows, :, lo], x[rows, :, hi] = u * cos - w * sin, w * cos + u * sin
            first += n
        first = 0
        for b, (n, a) in enumerate(zip(ql, past)):
            slot = torch.arange(a, a + n, device="cuda")
            to = s["block_table"][b].long()[slot // page]
            kc[to, slot % page] = k_new[first:first + n]
            vc[to, slot % page] = s["v"][first:first + n].double()
            first += n
        return {"q": q_new, "k_cache": kc, "v_cache": vc}
    if work(case)["flops"] > 4e12:
        return None
    G = case["q_heads"] // case["kv_heads"]
    outs, lses = [], []
    for b, (n, a) in enumerate(zip(ql, past)):
        if not n:
            continue
        pages = s["block_table"][b, :-(-(a + n) // page)].long()
        lo = max(0, a + 1 - case["window"]) if case["window"] else 0
        at = a + torch.arange(n, device="cuda")[:, None]
        key = torch.arange(lo, a + n, device="cuda")
        hidden = key > at
        if case["window"]:
            hidden |= key <= at - case["window"]
        out = torch.empty(n, case["q_heads"], case["dim"], dtype=torch.float64, device="cuda")
        lse = torch.empty(n, case["q_heads"], dtype=torch.float64, device="cuda")
        for h in range(case["kv_heads"]):
            k = s["k_cache"][pages, :, h].flatten(0, 1)[lo:a + n].double()
            v = s["v_cache"][pages, :, h].flatten(0, 1)[lo:a + n].double()
            for j in range(h * G, (h + 1) * G):
                x = (s["q"][first:first + n, j].double() @ k.T) * s["scale"]
                x = x.masked_fill(hidden, -math.inf)
                lse[:, j] = torch.logsumexp(x, -1)
                out[:, j] = torch.softmax(x, -1) @ v
        outs.append(out)
        lses.append(lse)
        first += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
