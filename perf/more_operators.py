"""Cases, plain forms and 64-bit values of the operators around a decoding step's forward:

- ``sample_tokens``: tokens drawn from rows of logits by given random numbers, with temperature, top-k, top-p and
  min-p, their log-probabilities, and the distribution they are drawn from (a drafter's q, as RAPID's verification
  takes it);
- ``paged_plan``: pages for a step's new tokens from a pool on the device, block tables, and the slot, position and
  request of every packed row;
- ``paged_kv_append`` with positions of several axes: keys and queries of text and images (time, height, width),
  each pair of a head turned by the position on its own axis, into the cache's pages.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One request's next draft: the latency of a call (the small vocabulary, fp32 logits).
        _sample("sample_b1_v32000", B=1, n=1, V=32000, type="f32", recipe="spiky", T=0.8, top_k=50, top_p=0.95),
        # An odd vocabulary, rows that start at odd addresses, a few positions to a request.
        _sample("sample_b5_odd_v4099", B=5, n=3, V=4099, type="bf16", recipe="zipf", T=1.3, top_p=0.8, min_p=0.02),
        # A draft for each of the 64 requests of the verification batch, nucleus only.
        _sample("sample_b64_v151936_top_p", B=64, n=1, V=151936, type="bf16", recipe="zipf", T=0.8, top_p=0.9),
        # Flat rows: the nucleus is tens of thousands of tokens.
        _sample("sample_b64_v151936_flat", B=64, n=1, V=151936, type="f32", recipe="spiky", T=1.0, top_p=0.95),
        # RAPID's drafter: 11 positions of 32 requests from the whole distribution, which the verification needs.
        _sample("sample_b32_n11_v128256_probs", B=32, n=11, V=128256, type="f32", recipe="ranked", T=1.0, probs=True),
        # A draft for 1024 requests, each with its own temperature and limits.
        _sample("sample_b1024_v151936_mixed", B=1024, n=1, V=151936, type="bf16", recipe="zipf", T=0.9, top_k=40,
                top_p=0.95, min_p=0.05, per_request=True),
        # The verification batch's step: 64 requests, K = 2.
        _plan("plan_b64_k2", B=64, new=(3, 3), past=(500, 12000), page=16),
        # 1024 requests, K = 8, some ended and their places taken by new prompts.
        _plan("plan_b1024_k8", B=1024, new=(9, 9), past=(1, 1000), page=32, released=0.06, prompt=(100, 2000)),
        # Long prompts all admitted at once.
        _plan("plan_b8_prompts", B=8, new=(1000, 8192), past=(0, 0), page=64, released=1.0, prompt=(1000, 8192)),
        # One token of one request appended behind text and an image.
        _axes("axes_decode_b1", B=1, q=(1, 1), past=(4095, 4095), heads=(32, 8), dim=128, page=16,
              axes=(16, 24, 24)),
        # Ten drafts and one for a batch, half precision, axes of neighbouring pairs in turns, part of the head turned.
        _axes("axes_verify_b32_g10", B=32, q=(11, 11), past=(300, 6000), heads=(28, 4), dim=128, page=32, type="f16",
              axes=(16, 8, 8), turns=True),
        # Prompts of text and images, written for the first time.
        _axes("axes_prompt_b6_images", B=6, q=(900, 7000), past=(0, 0), heads=(32, 8), dim=128, page=64,
              axes=(16, 24, 24), images=True),
    ]


def _sample(name, *, B, n, V, type, recipe, T=1.0, top_k=0, top_p=1.0, min_p=0.0, probs=False, per_request=False):
    return {"name": name, "op": "sample", "B": B, "n": n, "V": V, "type": type, "recipe": recipe, "T": T,
            "top_k": top_k, "top_p": top_p, "min_p": min_p, "probs": probs, "per_request": per_request}


def _plan(name, *, B, new, past, page, released=0.0, prompt=(1, 1), lens=1):
    return {"name": name, "op": "plan", "B": B, "new_lo": new[0], "new_hi": new[1], "past_lo": past[0],
            "past_hi": past[1], "page": page, "released": released, "prompt_lo": prompt[0], "prompt_hi": prompt[1],
            "lens": lens}


def _axes(name, *, B, q, past, heads, dim, page, axes, type="bf16", interleaved=False, turns=False, images=False,
          lens=1):
    return {"name": name, "op": "axes", "B": B, "q_lo": q[0], "q_hi": q[1], "past_lo": past[0], "past_hi": past[1],
            "q_heads": heads[0], "kv_heads": heads[1], "dim": dim, "page": page, "axis_t": axes[0], "axis_h": axes[1],
            "axis_w": axes[2], "type": type, "interleaved": interleaved, "turns": turns, "images": images,
            "lens": lens}


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    while True:
        op = rng.choice(["sample", "sample", "plan", "axes"])
        if op == "sample":
            case = _sample("", B=_log_int(rng, 1, 1024), n=rng.choice([1, 1, 1, 2, 3, 5, 11]),
                           V=rng.choice([_log_int(rng, 2, 200000), _log_int(rng, 1000, 160000), 32000, 128256, 151936]),
                           type=rng.choice(["bf16", "f32"]), recipe=rng.choice(["zipf", "zipf", "ranked", "spiky"]),
                           T=rng.choice([0.0, 0.3, 0.7, 1.0, 1.0, 1.5]),
                           top_k=rng.choice([0, 0, _log_int(rng, 1, 2000)]),
                           top_p=rng.choice([1.0, 0.5, 0.9, 0.95, 0.99]), min_p=rng.choice([0.0, 0.0, 0.02, 0.2]),
                           probs=rng.random() < 0.3, per_request=rng.random() < 0.3)
            if case["B"] * case["n"] * case["V"] * (3 if case["probs"] else 1) > 1.5e8:
                continue
        elif op == "plan":
            B = _log_int(rng, 1, 1500)
            k = rng.choice([1, 2, 3, 5, 9, 17])
            case = _plan("", B=B, new=rng.choice([(k, k), (0, k), (1, _log_int(rng, 2, 600))]),
                         past=(0, _log_int(rng, 1, 20000)), page=rng.choice([8, 16, 24, 32, 64, 128, 256]),
                         released=rng.choice([0.0, 0.05, 0.4, 1.0]), prompt=(0, _log_int(rng, 1, 9000)),
                         lens=rng.randrange(1 << 30))
            new, past, _, _ = _plan_lengths(case)
            if not sum(new) or sum(new) > 60000 or sum(past) > 4e6:
                continue
        else:
            kv_heads, group = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 3, 4, 7, 8])
            dim = rng.choice([64, 128, 128, 80, 96, 120])
            pairs = rng.choice([dim // 2, dim // 2, dim // 4])
            h = rng.randrange(0, pairs + 1)
            w = rng.randrange(0, pairs - h + 1)
            kind = rng.choice(["decode", "verify", "prompt"])
            past = (0, 0) if kind == "prompt" else (1, _log_int(rng, 64, 30000))
            k = {"decode": 1, "verify": rng.choice([3, 5, 9, 11])}.get(kind)
            case = _axes("", B=_log_int(rng, 1, 6 if kind == "prompt" else 200), past=past,
                         q=(k, k) if k else (1, _log_int(rng, 16, 6000)), heads=(kv_heads * group, kv_heads), dim=dim,
                         page=rng.choice([8, 16, 24, 32, 64, 128]), axes=(pairs - h - w, h, w),
                         type=rng.choice(["bf16", "f16"]), interleaved=rng.random() < 0.4, turns=rng.random() < 0.4,
                         images=kind == "prompt" and rng.random() < 0.7, lens=rng.randrange(1 << 30))
            ql, before = _lengths(case)
            if sum(ql) * dim * kv_heads * (group + 2) > 1.2e8 or 4 * kv_heads * dim * (sum(ql) + sum(before)) > 1.5e9:
                continue
        del case["name"]
        return case


def _spread(rng, lo, hi):
    if lo == hi:
        return lo
    return int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1)))) - 1 if lo == 0 else _log_int(rng, lo, hi)


def _lengths(case):
    """New tokens and tokens in the cache before them, per request."""
    rng = random.Random(case["lens"])
    B = case["B"]
    return [_spread(rng, case["q_lo"], case["q_hi"]) for _ in range(B)], \
        [_spread(rng, case["past_lo"], case["past_hi"]) for _ in range(B)]


def _plan_lengths(case):
    """New tokens, tokens in the cache, pages held, and whether the place's former request has ended, per request."""
    rng = random.Random(case["lens"])
    new, past, held, ended = [], [], [], []
    for _ in range(case["B"]):
        over = rng.random() < case["released"]
        before = _spread(rng, case["past_lo"], case["past_hi"])
        had = _spread(rng, case["prompt_lo"], case["prompt_hi"]) if over else before
        new.append(_spread(rng, case["prompt_lo"], case["prompt_hi"]) if over
                   else _spread(rng, case["new_lo"], case["new_hi"]))
        past.append(0 if over else before)
        held.append(-(-had // case["page"]))
        ended.append(over)
    return new, past, held, ended


def _axis_of_pairs(case):
    """The axis of every pair of a head: blocks, or neighbouring pairs in turns while an axis has pairs left."""
    left = [case["axis_t"], case["axis_h"], case["axis_w"]]
    if not case["turns"]:
        return [a for a in range(3) for _ in range(left[a])]
    out = []
    while sum(left):
        for a in range(3):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return out


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    return {"sample": _prepare_sample, "plan": _prepare_plan, "axes": _prepare_axes}[case["op"]](case, seed)


def _prepare_sample(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    B, n, V = case["B"], case["n"], case["V"]

    def exponential():
        return torch.empty(B, n, V, device=dev).exponential_(generator=g)

    if case["recipe"] == "zipf":      # a few tokens hold most of the mass: Gumbel noise over Zipf's ranks
        x = exponential().log_().mul_(-1.5).add_(exponential(), alpha=1.1)
    elif case["recipe"] == "ranked":  # normal noise over Zipf's ranks
        x = torch.randn(B, n, V, device=dev, generator=g).mul_(2.0).add_(exponential(), alpha=1.1)
    else:                             # five tokens stand out of a flat rest
        x = torch.randn(B, n, V, device=dev, generator=g).mul_(2.0)
        at = torch.randint(0, V, (B, n, 5), device=dev, generator=g)
        x.scatter_add_(2, at, torch.full(at.shape, 8.0, device=dev))
    f32 = dict(dtype=torch.float32, device=dev)
    s = {"op": "sample", "logits": x.to(_TYPES[case["type"]]), "u": torch.rand(B, n, device=dev, generator=g),
         "temperature": _f32(case["T"]), "top_k": case["top_k"], "top_p": _f32(case["top_p"]),
         "min_p": _f32(case["min_p"]), "tokens": torch.empty(B, n, dtype=torch.int32, device=dev),
         "logprobs": torch.empty(B, n, **f32),
         "probs": torch.empty(B, n, V, **f32) if case["probs"] else None,
         "status": torch.zeros(B, dtype=torch.int32, device=dev)}
    if case["per_request"]:
        r = random.Random(seed)
        pick = lambda *of: [r.choice(of) for _ in range(B)]
        s["temperature"] = torch.tensor([t * case["T"] for t in pick(0.0, 0.6, 1.0, 1.2)], **f32)
        s["top_k"] = torch.tensor([int(f * case["top_k"]) for f in pick(0, 0.5, 1, 2)], dtype=torch.int32, device=dev)
        s["top_p"] = torch.tensor([min(1.0, f * case["top_p"]) for f in pick(0.8, 1.0, 2.0)], **f32)
        s["min_p"] = torch.tensor([f * case["min_p"] for f in pick(0.0, 1.0, 2.0)], **f32)
    return s


def _f32(x):
    """x as a number of 32 bits holds it."""
    return float(torch.tensor(x, dtype=torch.float32))


def _prepare_plan(case, seed):
    dev = "cuda"
    new, past, held, ended = _plan_lengths(case)
    B, page, N = case["B"], case["page"], sum(new)
    need = [max(0, -(-(a + k) // page) - (0 if e else h)) for a, k, h, e in zip(past, new, held, ended)]
    width = max(max(held), max(-(-(a + k) // page) for a, k in zip(past, new)), 1) + 1
    n_pages = sum(held) + sum(need) + 5
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table, at = [], 0
    for h in held:
        table.append(order[at:at + h] + [-1] * (width - h))
        at += h
    i32 = dict(dtype=torch.int32, device=dev)
    free = order[at:] + [-1] * at
    return {"op": "plan", "cache_len": torch.tensor(past, **i32), "new_len": torch.tensor(new, **i32),
            "block_table": torch.tensor(table, **i32), "held": torch.tensor(held, **i32),
            "free_pages": torch.tensor(free, **i32), "free_count": torch.tensor([n_pages - at], **i32),
            "release": torch.tensor(ended, device=dev), "page": page, "indptr": torch.empty(B + 1, **i32),
            "slots": torch.empty(N, dtype=torch.int64, device=dev), "positions": torch.empty(N, **i32),
            "requests": torch.empty(N, **i32), "status": torch.zeros(B, **i32)}


def _prepare_axes(case, seed):
    dev, dt = "cuda", _TYPES[case["type"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    ql, past = _lengths(case)
    B, Hq, Hkv, D, page = case["B"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    N = sum(ql)
    pages = [-(-(a + b) // page) for a, b in zip(ql, past)]
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table, at = [], 0
    for k in pages:
        table.append(order[at:at + k] + [-1] * (max(max(pages), 1) - k))
        at += k
    starts = [0]
    for k in ql:
        starts.append(starts[-1] + k)
    pos = torch.cat([_positions(case, n, a, b) for b, (n, a) in enumerate(zip(ql, past))] or
                    [torch.zeros(3, 0, dtype=torch.int64)], 1)
    axes = _axis_of_pairs(case)
    R = 2 * len(axes)
    i32 = dict(dtype=torch.int32, device=dev)
    limit = int(pos.max()) + 1 if N else 1
    angle = torch.arange(limit, dtype=torch.float64, device=dev)[:, None] \
        * 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=dev) / R)
    # q, k and v are views of one projection's output, as a model makes them
    qkv = torch.randn(N, (Hq + 2 * Hkv) * D, dtype=dt, device=dev, generator=g)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1))
    return {"op": "axes", "q": q, "k": k, "v": v, "rotary": torch.cat([angle.cos(), angle.sin()], 1).float(),
            "k_cache": torch.randn(n_pages, page, Hkv, D, dtype=dt, device=dev, generator=g),
            "v_cache": torch.randn(n_pages, page, Hkv, D, dtype=dt, device=dev, generator=g),
            "block_table": torch.tensor(table, **i32), "cache_len": torch.tensor(past, **i32),
            "indptr": torch.tensor(starts, **i32), "positions": pos.to(**i32), "axes": bytes(axes),
            "interleaved": case["interleaved"], "q_out": torch.empty(N, Hq, D, dtype=dt, device=dev),
            "status": torch.zeros(B, **i32)}


def _positions(case, n, past, b):
    """[3, n]: a chunk's positions on the axes.  Text counts up on all three; an image takes one step in time, its
    rows and columns count from there, and what follows starts behind the larger of the two."""
    rng = random.Random(case["lens"] * 1000003 + b)
    at = past - past // 3 if past else 0  # (an image in the cache has taken fewer positions than slots)
    parts, left = [], n
    while left:
        h, w = rng.randrange(8, 40), rng.randrange(8, 40)
        text = min(left, rng.randrange(20, 200)) if case["images"] else left
        parts.append(torch.arange(at, at + text).expand(3, text))
        at, left = at + text, left - text
        if case["images"] and left:
            size = min(left, h * w)
            i = torch.arange(size)
            parts.append(at + torch.stack([torch.zeros_like(i), i // w, i % w]))
            at, left = at + max(h, w), left - size
    return torch.cat(parts, 1) if parts else torch.zeros(3, 0, dtype=torch.int64)


# ------------------------------------------------------------------ one pass

def run(s):
    if not own:
        return {"sample": _sample_plain, "plan": _plan_plain, "axes": _axes_plain}[s["op"]](s)
    import speculative_decoding_logit_gb300 as asv
    if s["op"] == "sample":
        out = asv.SampleOutput(s["tokens"], s["logprobs"], s["probs"], s["status"])
        asv.sample_tokens(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                          min_p=s["min_p"], out=out)
        return {k: v for k, v in (("tokens", out.tokens), ("logprobs", out.logprobs), ("probs", out.probs))
                if v is not None}
    if s["op"] == "plan":
        out = asv.PagedPlanOutput(s["indptr"], s["slots"], s["positions"], s["requests"], s["status"])
        asv.paged_plan(s["cache_len"], s["new_len"], s["block_table"], s["held"], s["free_pages"], s["free_count"],
                       s["page"], release=s["release"], out=out)
        return _planned(s)
    out = asv.PagedAppendOutput(s["q_out"], s["status"])
    asv.paged_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["cache_len"], s["indptr"],
                        q=s["q"], rotary=s["rotary"], interleaved=s["interleaved"], positions=s["positions"],
                        axes=s["axes"], out=out)
    return {"q": out.q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _planned(s):
    return {k: s[k] for k in ("indptr", "slots", "positions", "requests", "block_table", "held", "free_pages",
                              "free_count")}


def _sample_plain(s):
    B, n, V = s["logits"].shape

    def column(x, dtype):  # a parameter for each row
        x = x.to(dtype) if isinstance(x, torch.Tensor) else torch.full((B,), x, dtype=dtype, device="cuda")
        return x.repeat_interleave(n)[:, None]

    logits, u = s["logits"].reshape(B * n, V), s["u"].reshape(-1, 1).double()
    T, p, least = (column(s[k], torch.float64) for k in ("temperature", "top_p", "min_p"))
    k = column(s["top_k"], torch.int64)
    tokens, logs, probs = [], [], []
    # sums of 64 bits: a nucleus' border and a draw's are next to values that 32 bits do not tell apart
    step = max(1, (1 << 26) // V)
    for r in range(0, B * n, step):
        rows = slice(r, r + step)
        x, at = logits[rows].float().sort(dim=1, descending=True, stable=True)
        greedy = T[rows] == 0
        w = ((x.double() - x[:, :1].double()) / torch.where(greedy, 1.0, T[rows])).exp()
        place = torch.arange(V, device="cuda")
        keep = (place < k[rows]) | (k[rows] <= 0)
        w *= keep
        total = w.cumsum(1)
        nucleus = (total - w < p[rows] * total[:, -1:]) | (p[rows] >= 1)
        keep &= (nucleus & (w >= least[rows]) & ~greedy) | (place == 0)
        w = torch.zeros_like(w).scatter_(1, at, w * keep)
        total = w.cumsum(1)
        drawn = (total <= u[rows] * total[:, -1:]).sum(1, keepdim=True).clamp(max=V - 1)
        drawn = torch.where(greedy, at[:, :1], drawn)
        tokens.append(drawn.to(torch.int32))
        logs.append((w.gather(1, drawn) / total[:, -1:]).log().float())
        if s["probs"] is not None:
            probs.append((w / total[:, -1:]).float())
    out = {"tokens": torch.cat(tokens).reshape(B, n), "logprobs": torch.cat(logs).reshape(B, n)}
    if s["probs"] is not None:
        out["probs"] = torch.cat(probs).reshape(B, n, V)
    return out


def _plan_plain(s):
    page, table, free, N = s["page"], s["block_table"], s["free_pages"], s["slots"].shape[0]
    B, width = table.shape
    past, new, held = s["cache_len"].long(), s["new_len"].long(), s["held"].long()
    entry = torch.arange(width, device="cuda")
    # pages of requests that have ended, onto the pool
    back = torch.where(s["release"], held, 0)
    count = s["free_count"].long()
    place = count + (back.cumsum(0) - back)[:, None] + entry
    ended = entry < back[:, None]
    free[place[ended]] = table[ended]
    table.masked_fill_(ended, -1)
    held, count = held - back, count + back.sum()
    # pages that the new tokens need, from its top
    need = (-(-(past + new) // page) - held).clamp(min=0)
    fits = ((need.cumsum(0) <= count) | (need == 0)) & (new.cumsum(0) <= N)
    need, new = torch.where(fits, need, 0), torch.where(fits, new, 0)
    taken = (entry >= held[:, None]) & (entry < (held + need)[:, None])
    place = (count - 1 - (need.cumsum(0) - need))[:, None] - (entry - held[:, None])
    table[taken] = free[place[taken]]
    s["held"].copy_(held + need)
    s["free_count"].copy_(count - need.sum())
    start = new.cumsum(0)
    s["indptr"][0] = 0
    s["indptr"][1:] = start
    row = torch.arange(N, device="cuda")
    request = torch.searchsorted(start, row, right=True).clamp(max=B - 1)
    at = past[request] + row - (start - new)[request]
    there = row < start[-1]
    entry = (at // page).clamp(0, width - 1)
    s["slots"].copy_(torch.where(there, table[request, entry].long() * page + at % page, -1))
    s["positions"].copy_(torch.where(there, at, -1))
    s["requests"].copy_(torch.where(there, request, -1))
    return _planned(s)


def _axes_plain(s):
    row = torch.arange(s["k"].shape[0], device="cuda")
    request = torch.searchsorted(s["indptr"][1:].long(), row, right=True)
    at = s["cache_len"].long()[request] + row - s["indptr"].long()[request]
    page = s["k_cache"].shape[1]
    to = s["block_table"].long()[request, at // page], at % page
    axis = torch.tensor(list(s["axes"]), device="cuda")
    half = axis.shape[0]
    pair = torch.arange(half, device="cuda")
    place = s["positions"].long()[axis].T                 # [N, pairs]
    cos, sin = s["rotary"][place, pair][:, None], s["rotary"][place, half + pair][:, None]
    s["k_cache"][to] = _turn_plain(s["k"], cos, sin, s["interleaved"])
    s["v_cache"][to] = s["v"]
    return {"q": _turn_plain(s["q"], cos, sin, s["interleaved"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _turn_plain(x, cos, sin, interleaved):
    R = 2 * cos.shape[-1]
    y, turned = x.float(), x[..., :R].float()
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :R // 2], turned[..., R // 2:])
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)
    return torch.cat([turned, y[..., R:]], -1).to(x.dtype)


# ------------------------------------------------------------------ floors and 64-bit values

def work(case):
    if case["op"] == "sample":
        rows, V = case["B"] * case["n"], case["V"]
        size = 2 if case["type"] == "bf16" else 4
        moved = rows * V * (size + (4 if case["probs"] else 0)) + 12 * rows
        return {"bytes": moved + (16 * case["B"] if case["per_request"] else 0), "flops": 4 * rows * V}
    if case["op"] == "plan":
        new, past, held, ended = _plan_lengths(case)
        page, N, B = case["page"], sum(new), case["B"]
        back = sum(h for h, e in zip(held, ended) if e)
        need = sum(max(0, -(-(a + k) // page) - (0 if e else h)) for a, k, h, e in zip(past, new, held, ended))
        entries = sum(-(-(a + k) // page) - a // page for a, k in zip(past, new) if k)
        return {"bytes": N * 16 + B * 21 + 12 * back + 8 * need + 4 * entries, "flops": 0}
    ql, past = _lengths(case)
    Hq, Hkv, D, N = case["q_heads"], case["kv_heads"], case["dim"], sum(ql)
    pairs = case["axis_t"], case["axis_h"], case["axis_w"]
    at = torch.cat([_positions(case, n, a, b) for b, (n, a) in enumerate(zip(ql, past))], 1)
    table = sum(8 * pairs[i] * at[i].unique().numel() for i in range(3))
    moved = 2 * 2 * N * (Hq + 2 * Hkv) * D + table + 4 * 3 * N + 4 * (2 * case["B"] + N)
    return {"bytes": moved, "flops": 3 * N * (Hq + Hkv) * 2 * sum(pairs)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"sample": _sample_exact, "plan": _plan_exact, "axes": _axes_exact}[case["op"]](case, s)


def _sample_exact(case, s):
    if case["B"] * case["n"] * case["V"] > 2.5e8:
        return None
    B, n, V = s["logits"].shape
    value = lambda x, b: float(x[b]) if isinstance(x, torch.Tensor) else x
    host = {k: s[k].cpu() if isinstance(s[k], torch.Tensor) else s[k] for k in ("temperature", "top_k", "top_p", "min_p")}
    tokens = torch.empty(B, n, dtype=torch.int32, device="cuda")
    logs = torch.zeros(B, n, dtype=torch.float64, device="cuda")
    probs = torch.empty(B, n, V, dtype=torch.float64, device="cuda") if s["probs"] is not None else None
    for b in range(B):
        T, k, p, least = (value(host[x], b) for x in ("temperature", "top_k", "top_p", "min_p"))
        for i in range(n):
            x = s["logits"][b, i].double()
            # from the smallest up, the highest index first among equals: the order turned round
            up = torch.flip(x, (0,)).argsort(stable=True)
            order = (V - 1 - up).flip(0)
            if T == 0:
                tokens[b, i] = order[0]
                if probs is not None:
                    probs[b, i] = 0
                    probs[b, i, order[0]] = 1
                continue
            if k > 0:
                order = order[:int(k)]
            share = torch.softmax(x[order] / T, 0)
            after = share.flip(0).cumsum(0).flip(0)       # from each on to the last
            count = order.shape[0] if p >= 1 else int((after > 1 - p).sum())
            if least > 0:
                count = min(count, int((share >= least * share[0]).sum()))
            kept = order[:max(count, 1)]
            mass = torch.zeros(V, dtype=torch.float64, device="cuda")
            log = torch.log_softmax(x[kept] / T, 0)
            mass[kept] = log.exp()
            below = mass.cumsum(0)
            tokens[b, i] = torch.searchsorted(below, s["u"][b, i].double() * below[-1], right=True).clamp(max=V - 1)
            logs[b, i] = log[kept == tokens[b, i]][0]
            if probs is not None:
                probs[b, i] = mass
    out = {"tokens": tokens, "logprobs": logs}
    return out if probs is None else out | {"probs": probs}


def _plan_exact(case, s):
    page, N = s["page"], s["slots"].shape[0]
    table, pool = s["block_table"].tolist(), s["free_pages"].tolist()
    held, top = s["held"].tolist(), int(s["free_count"])
    past, new, ended = s["cache_len"].tolist(), s["new_len"].tolist(), s["release"].tolist()
    for b in range(case["B"]):
        if ended[b]:
            for j in range(held[b]):
                pool[top], table[b][j] = table[b][j], -1
                top += 1
            held[b] = 0
    room, asked, rows = top, 0, 0
    slots, positions, requests, indptr = [], [], [], [0]
    for b in range(case["B"]):
        need = max(0, -(-(past[b] + new[b]) // page) - held[b])
        asked, rows = asked + need, rows + new[b]
        if (need == 0 or asked <= room) and rows <= N:
            for _ in range(need):
                top -= 1
                table[b][held[b]] = pool[top]
                held[b] += 1
            for at in range(past[b], past[b] + new[b]):
                slots.append(table[b][at // page] * page + at % page)
                positions.append(at)
                requests.append(b)
        indptr.append(len(slots))
    rest = [-1] * (N - len(slots))
    out = {"indptr": indptr, "slots": slots + rest, "positions": positions + rest, "requests": requests + rest,
           "block_table": table, "held": held, "free_pages": pool, "free_count": [top]}
    return {k: torch.tensor(v, dtype=s[k].dtype, device="cuda") for k, v in out.items()}


def _axes_exact(case, s):
    kc, vc, q_new, k_new = s["k_cache"].double(), s["v_cache"].double(), s["q"].double(), s["k"].double()
    ql, past = _lengths(case)
    half, rotary, where = len(s["axes"]), s["rotary"].double(), s["positions"].long()
    for j, axis in enumerate(s["axes"]):
        lo, hi = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + half)
        cos, sin = rotary[where[axis], j][:, None], rotary[where[axis], half + j][:, None]
        for x in (q_new, k_new):
            u, w = x[:, :, lo].clone(), x[:, :, hi].clone()
            x[:, :, lo], x[:, :, hi] = u * cos - w * sin, w * cos + u * sin
    first = 0
    for b, (n, a) in enumerate(zip(ql, past)):
        slot = torch.arange(a, a + n, device="cuda")
        to = s["block_table"][b].long()[slot // case["page"]]
        kc[to, slot % case["page"]] = k_new[first:first + n]
        vc[to, slot % case["page"]] = s["v"][first:first + n].double()
        first += n
    return {"q": q_new, "k_cache": kc, "v_cache": vc}
