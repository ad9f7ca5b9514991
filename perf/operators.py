"""The decode step around the expert layer: routing, the paged 8-bit cache, attention over it.

Four operators, each as plain torch arithmetic (``own = False``) and as the
library's call (``own = True``):

* ``route``: router logits -> the top-k expert ids and weights of each token;
* ``plan``: request lengths -> block-table entries, sequence lengths, token
  positions and cache slots;
* ``append``: new key and value rows -> e4m3 codes in the cache, one
  power-of-two scale for each page and head;
* ``attend``: causal attention of the new tokens over the cache.

The cache is uint8 [pages, kv_heads, page, head_dim] of e4m3 codes for keys and
another for values, with uint8 [pages, kv_heads] E8M0 scales (byte b stands
for 2^(b - 127)).
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
WORKSPACE_BYTES = 32 << 20  # what an attend call may need between its CTAs
LARGEST = {"bytes": 5.3e8, "flops": 1.6e11}  # the largest listed cases' work


# ------------------------------------------------------------------ the cases
def listed():
    route = dict(op="route", experts=384, topk=16, dtype="float32", scoring="sigmoid", bias=True, groups=1,
                 group_topk=1, group_score=1, renormalize=True, scale=1.0)
    plan = dict(op="plan", page=64, low=1, empty_every=0, pad=0)
    append = dict(op="append", page=64, kv_heads=8, head_dim=128, low=1, empty_every=0, pad=0)
    attend = dict(op="attend", page=64, q_heads=64, kv_heads=8, head_dim=128, window=0, empty_every=0, pad=0)
    return [
        # One token of the 384-expert, top-16 layer: latency alone.
        dict(route, name="route_single", tokens=1),
        # A decode batch whose logits come out of a BF16 product, softmax scores.
        dict(route, name="route_batch_softmax", tokens=64, dtype="bfloat16", scoring="softmax", bias=False),
        # A ragged prompt through a router limited to half of its expert groups.
        dict(route, name="route_prompt_groups", tokens=16381, groups=8, group_topk=4, group_score=2, scale=2.5),
        # The slots of one decode step: one new token for each of 64 requests.
        dict(plan, name="plan_decode", requests=64, context=8192, query=1),
        # Prompts that arrive in a large queue, small pages, a padded token axis.
        dict(plan, name="plan_prompts", requests=1000, context=3000, query=400, page=16, pad=512, empty_every=9),
        # The cache write of one decode step.
        dict(append, name="append_decode", requests=64, context=1024, query=1),
        # The cache write of whole prompts, their lengths odd.
        dict(append, name="append_prompts", requests=11, context=1, query=1500),
        # One request, a short context: latency alone.
        dict(attend, name="attend_single", requests=1, low=777, context=777, query=1),
        # A decode batch of ragged contexts: the memory-bound middle of serving.
        dict(attend, name="attend_batch", requests=64, low=1, context=8192, query=1),
        # Two requests with long contexts, 28 heads of 128 (the hidden size 3584) on 4, so 7 share one.
        dict(attend, name="attend_long", requests=2, low=100001, context=131071, query=1, page=128, q_heads=28,
             kv_heads=4),
        # Four to eight drafted tokens verified at once, a sliding window, some slots of the batch empty.
        dict(attend, name="attend_verify_window", requests=40, low=5, context=6000, query=8, page=16, q_heads=24,
             kv_heads=8, head_dim=64, window=1024, empty_every=7, pad=3),
        # Two prompt chunks over a cache that holds their earlier parts.
        dict(attend, name="attend_chunk", requests=2, low=4001, context=6001, query=700),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    while True:
        case = _draw(rng)
        w = work(case)
        if w["bytes"] <= LARGEST["bytes"] and w["flops"] <= LARGEST["flops"] and plain_bytes(case) <= 9e9:
            return case


def _draw(rng):
    op = rng.choice(["route", "plan", "append", "attend", "attend"])
    if op == "route":
        experts = _log(rng, 8, 1024)
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if experts % g == 0 and experts // g >= 2])
        group_topk = rng.randint(1, groups)
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=experts,
                    topk=rng.randint(1, min(32, group_topk * (experts // groups))),
                    dtype=rng.choice(["float32", "bfloat16", "float16"]), scoring=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, group_topk=group_topk, group_score=rng.choice([1, 2]),
                    renormalize=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))
    lengths = dict(requests=_log(rng, 1, 64), low=1, context=_log(rng, 1, 16384),
                   query=rng.choice([1, 1, rng.randint(2, 9), _log(rng, 2, 900)]),
                   page=rng.choice([16, 32, 64, 128]), empty_every=rng.choice([0, 0, 5]), pad=rng.choice([0, 0, 7]))
    if op == "plan":
        lengths["requests"] = _log(rng, 1, 1024)
        return dict(op=op, **lengths)
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    cache = dict(kv_heads=kv_heads, head_dim=rng.choice([64, 128, 128, 256]))
    if op == "append":
        return dict(op=op, **lengths, **cache)
    return dict(op=op, **lengths, **cache, q_heads=kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 16]),
                window=rng.choice([0, 0, _log(rng, 1, 4096)]))


# ---------------------------------------------------------------- the lengths
def lengths_of(case):
    """(cached tokens, new tokens) of each request, from the case alone: two golden-ratio-like sequences over the range."""
    cached, new = [], []
    for i in range(case["requests"]):
        u, w = ((i + 1) * 0.6180339887) % 1.0, ((i + 1) * 0.4142135624) % 1.0
        empty = case["empty_every"] and i % case["empty_every"] == case["empty_every"] - 1
        q = 1 if case["query"] == 1 else case["query"] // 2 + 1 + int(u * (case["query"] - case["query"] // 2 - 1))
        low = min(case["low"], case["context"])
        total = low + int(round((case["context"] - low) * w))
        # A decode context holds the new tokens; a prompt (context below them) starts the cache.
        cached.append(0 if empty else max(0, total - q))
        new.append(0 if empty else q)
    return cached, new


def visible(case):
    """(tokens of the cache that some query sees, query-key pairs) over the requests."""
    tokens = pairs = 0
    for c, q in zip(*lengths_of(case)):
        w = case["window"] or c + q
        tokens += min(c + q, w + q - 1) if q else 0
        pairs += sum(min(c + i + 1, w) for i in range(q))
    return tokens, pairs


def work(case):
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": t * (e * size + case["topk"] * 8) + (4 * e if case["bias"] else 0), "flops": 4 * t * e}
    cached, new = lengths_of(case)
    tokens = sum(new)
    if case["op"] == "plan":
        pages = sum(-(-(c + q) // case["page"]) + -(-c // case["page"]) * -1 for c, q in zip(cached, new))
        return {"bytes": 16 * case["requests"] + 12 * (tokens + case["pad"]) + 8 * pages, "flops": 0}
    row = case["kv_heads"] * case["head_dim"]
    if case["op"] == "append":
        return {"bytes": 2 * tokens * row * 3 + 8 * (tokens + case["pad"]), "flops": 4 * tokens * row}
    seen, pairs = visible(case)
    out = tokens * case["q_heads"] * (case["head_dim"] * 4 + 4)
    return {"bytes": 2 * seen * row + 2 * (seen // case["page"]) * case["kv_heads"] + out,
            "flops": 4 * pairs * case["q_heads"] * case["head_dim"]}


def plain_bytes(case):
    """About what the plain form holds at once (its gathered, padded keys, values and scores in 32 bits)."""
    if case["op"] != "attend":
        return 0
    cached, new = lengths_of(case)
    longest = max(c + q for c, q in zip(cached, new)) + case["page"]
    return 4 * case["requests"] * longest * (4 * case["kv_heads"] * case["head_dim"] + 4 * max(new) * case["q_heads"])


# ----------------------------------------------------------------- the inputs
def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    s = dict(case=dict(case))
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        popular = 0.7 * torch.randn(e, generator=g, device=DEVICE)
        logits = torch.randn(t, e, generator=g, device=DEVICE) * 1.2 + popular
        s["logits"] = logits.to(getattr(torch, case["dtype"]))
        # A balance bias moves by a fixed step at each update.
        steps = torch.randint(-60, 61, (e,), generator=g, device=DEVICE)
        s["bias"] = steps.float() * 0.001 if case["bias"] else None
        s["ids"] = torch.empty(t, k, dtype=torch.int32, device=DEVICE)
        s["weights"] = torch.empty(t, k, dtype=torch.float32, device=DEVICE)
        return s
    cached, new = lengths_of(case)
    order = torch.randperm(len(new), generator=torch.Generator().manual_seed(seed)).tolist()
    cached, new = [cached[i] for i in order], [new[i] for i in order]
    page, requests, tokens = case["page"], len(new), sum(new) + case["pad"]
    held = [-(-c // page) for c in cached]
    total = [-(-(c + q) // page) for c, q in zip(cached, new)]
    pool = sum(total) + 5
    ids = torch.randperm(pool, generator=g, device=DEVICE).int()
    # The table holds the pages of the cached tokens; the free list has the rest.
    width = max(max(total), 1) + 1
    held_t = torch.tensor(held, device=DEVICE)
    at = torch.arange(width, device=DEVICE)
    start = torch.cumsum(held_t, 0) - held_t
    table = torch.where(at < held_t[:, None], ids[(start[:, None] + at).clamp(max=pool - 1)], -1)
    free = ids[sum(held):].contiguous()

    def ints(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device=DEVICE)

    s.update(context_lens=ints(cached), query_lens=ints(new), page=page, requests=requests, tokens=tokens,
             table=table.int().contiguous(), free=free, free_head=ints([0]),
             query_start=torch.empty(requests + 1, dtype=torch.int32, device=DEVICE),
             seq_lens=torch.empty(requests, dtype=torch.int32, device=DEVICE),
             positions=torch.empty(tokens, dtype=torch.int32, device=DEVICE),
             slots=torch.empty(tokens, dtype=torch.int64, device=DEVICE),
             counts=torch.empty(4, dtype=torch.int32, device=DEVICE))
    if case["op"] == "plan":
        return s
    # The step's plan, which every layer's append and attend calls share.
    p = plan_plain(s)
    s["table"], s["query_start"], s["seq_lens"], s["slots"] = p["table"], p["query_start"], p["seq_lens"], p["slots"]
    heads, dim = case["kv_heads"], case["head_dim"]
    s["cache"] = codes(pool, heads, page, dim, g) + codes(pool, heads, page, dim, g)
    s["cache"] = (s["cache"][0], s["cache"][2], s["cache"][1], s["cache"][3])  # k, v, k_scale, v_scale
    if case["op"] == "append":
        # One projection gives a token's keys and values side by side; some channels are larger than others.
        kv = torch.randn(tokens, 2, heads, dim, generator=g, device=DEVICE)
        kv *= 1 + 3 * (torch.rand(2, heads, dim, generator=g, device=DEVICE) > 0.97)
        kv = kv.to(torch.bfloat16)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        return s
    s["q"] = torch.randn(tokens, case["q_heads"], dim, generator=g, device=DEVICE).to(torch.bfloat16)
    s["scale"] = 1.0 / math.sqrt(dim)
    s["longest_query"] = max(max(new), 1)
    s["out"] = torch.zeros(tokens, case["q_heads"], dim, dtype=torch.bfloat16, device=DEVICE)
    s["lse"] = torch.zeros(tokens, case["q_heads"], dtype=torch.float32, device=DEVICE)
    s["workspace"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device=DEVICE)
    return s


def codes(pool, heads, page, dim, g):
    """e4m3 codes as a cache of unit normals has them, with scales that differ by page and head."""
    data = torch.empty(pool, heads, page, dim, dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 26) // (heads * page * dim))
    for i in range(0, pool, step):
        part = torch.randn(data[i:i + step].shape, generator=g, device=DEVICE)
        data[i:i + step] = (part * 90).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return data, torch.randint(119, 122, (pool, heads), generator=g, device=DEVICE, dtype=torch.uint8)


# ------------------------------------------------------------ one pass through
def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": route_own, "plan": plan_own, "append": append_own, "attend": attend_own}[op](state)
    return {"route": route_plain, "plan": plan_plain, "append": append_plain, "attend": attend_plain}[op](state)


def route_own(s):
    import mxfp4_weight_mxfp8_gb300 as moe

    c = s["case"]
    moe.moe_route(s["logits"], s["ids"], s["weights"],
                  scoring=moe.SCORE_SIGMOID if c["scoring"] == "sigmoid" else moe.SCORE_SOFTMAX, bias=s["bias"],
                  groups=c["groups"], group_topk=c["group_topk"], group_score=c["group_score"],
                  renormalize=c["renormalize"], scale=c["scale"])
    return {"ids": s["ids"], "weights": s["weights"]}


def plan_own(s):
    import mxfp4_weight_mxfp8_gb300 as moe

    moe.moe_kv_plan(s["context_lens"], s["query_lens"], s["page"], s["table"], s["free"], s["free_head"],
                    s["query_start"], s["seq_lens"], s["positions"], s["slots"], s["counts"])
    return {n: s[n] for n in ("table", "query_start", "seq_lens", "positions", "slots", "counts")}


def append_own(s):
    import mxfp4_weight_mxfp8_gb300 as moe

    moe.moe_kv_append(s["cache"], s["k"], s["v"], s["slots"])
    return cache_values(s["cache"])


def attend_own(s):
    import mxfp4_weight_mxfp8_gb300 as moe

    moe.moe_kv_attend(s["cache"], s["q"], s["table"], s["query_start"], s["seq_lens"], s["out"], s["workspace"],
                      lse=s["lse"], scale=s["scale"], window=s["case"]["window"])
    return {"out": s["out"], "lse": s["lse"]}


def cache_values(cache):
    """The cache as the numbers that its codes stand for, next to their exponents."""
    k, v, ks, vs = cache
    return {"k": k.view(torch.float8_e4m3fn), "v": v.view(torch.float8_e4m3fn), "k_scale": ks, "v_scale": vs}


# -------------------------------------------------------------- the plain form
def tree_sum(x):
    """Sum over the last axis, halving it: element i and i + n/2 first, over 1024 places."""
    x = torch.nn.functional.pad(x, (0, 1024 - x.shape[-1]))
    while x.shape[-1] > 1:
        x = x[..., : x.shape[-1] // 2] + x[..., x.shape[-1] // 2:]
    return x


def route_plain(s):
    c, x = s["case"], s["logits"].float()
    lowest = -math.inf
    masked = torch.isnan(x) | (x == lowest)
    if c["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        x = x.clamp(-3.4028234663852886e38, 3.4028234663852886e38)
        top = torch.where(masked, lowest, x).amax(-1, keepdim=True)
        e = torch.where(masked, 0.0, torch.exp(x - top))
        score = e / tree_sum(e)
    if s["bias"] is not None:
        key = score + s["bias"]
    else:  # both scores grow with the logit: where scores are only compared, the logits are
        key = score if c["groups"] > 1 and c["group_score"] == 2 else x
    key = torch.where(masked | torch.isnan(key), lowest, key)
    if c["groups"] > 1:
        by_group = key.view(key.shape[0], c["groups"], -1)
        best = by_group.sort(dim=-1, descending=True).values[..., : c["group_score"]]
        group = best[..., 0] if c["group_score"] == 1 else best[..., 0] + best[..., 1]
        order = group.sort(dim=-1, descending=True, stable=True).indices[:, : c["group_topk"]]
        kept = torch.zeros_like(group, dtype=torch.bool).scatter_(1, order, True)
        key = torch.where(kept[..., None], by_group, lowest).view_as(key)
    keys, ids = (v[:, : c["topk"]] for v in key.sort(dim=-1, descending=True, stable=True))
    w = torch.where(keys == lowest, 0.0, score.gather(1, ids))
    if c["renormalize"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return {"ids": ids.int(), "weights": w * c["scale"]}


def plan_plain(s):
    page, width, tokens = s["page"], s["table"].shape[1], s["tokens"]
    cached, new = s["context_lens"].long(), s["query_lens"].long()
    seq = cached + new
    ends = torch.cumsum(new, 0)
    query_start = torch.nn.functional.pad(ends, (1, 0))
    held, needed = (cached + page - 1) // page, (seq + page - 1) // page
    grown = torch.cumsum(needed - held, 0)
    # Page `at` of request r: the table's own below `held`, then the free list's in request order.
    at = torch.arange(width, device=seq.device)
    rank = s["free_head"].long() + (grown - (needed - held))[:, None] + at - held[:, None]
    taken = (at >= held[:, None]) & (at < needed[:, None])
    fresh = torch.where(rank < s["free"].numel(), s["free"][rank.clamp(0, s["free"].numel() - 1)], -1)
    table = torch.where(taken, fresh, s["table"])
    t = torch.arange(tokens, device=seq.device)
    r = torch.searchsorted(ends, t, right=True).clamp(max=seq.numel() - 1)
    used = t < ends[-1]
    pos = cached[r] + t - query_start[r]
    owner = table[r, (pos // page).clamp(0, width - 1)].long()
    slots = torch.where(used & (owner >= 0), owner * page + pos % page, -1)
    counts = torch.stack([ends[-1], s["free_head"][0].long() + grown[-1], seq.max(), torch.zeros_like(seq[0])])
    return {"table": table.int(), "query_start": query_start.int(), "seq_lens": seq.int(),
            "positions": torch.where(used, pos, 0).int(), "slots": slots, "counts": counts.int()}


def power(e):
    """2^e in 32 bits, exactly, for whole e in [-127, 127]."""
    e = e.int()
    return torch.where(e > -127, (e + 127) << 23, 0x00400000).view(torch.float32)


def exponent(amax):
    """The smallest E with amax <= 448 * 2^E, at least -127; -127 for zero and what 32 bits hold without a leading one."""
    m, e = torch.frexp(amax)
    return torch.where(amax >= 2.0 ** -126, e - 9 + (m > 0.875).int(), -127).clamp(-127, 127).int()


def append_plain(s):
    k, v, ks, vs = s["cache"]
    page = k.shape[2]
    used = s["slots"] >= 0
    owner = torch.where(used, s["slots"] // page, k.shape[0])  # unused rows go to a page past the last
    off = s["slots"] % page
    first = torch.full((k.shape[0] + 1,), page, device=k.device).scatter_reduce_(0, owner, off, "amin")[:-1]
    touched = (first < page)[:, None]
    live = (first > 0)[:, None]
    append_rows(s["k"].float(), k, ks, owner, off, used, first, touched, live)
    append_rows(s["v"].float(), v, vs, owner, off, used, first, touched, live)
    return cache_values(s["cache"])


def append_rows(x, cache, scale, owner, off, used, first, touched, live):
    pages, heads, page, dim = cache.shape
    amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    need = torch.full((pages + 1, heads), -127, dtype=torch.int32, device=x.device)
    need.scatter_reduce_(0, owner[:, None].expand(-1, heads), exponent(amax), "amax")
    old = scale.int() - 127
    new = torch.where(touched, torch.where(live, torch.maximum(need[:-1], old), need[:-1]), old)
    # Earlier tokens of a page whose scale grows are rounded again to the new one.
    moved = touched & live & (new > old)
    before = torch.arange(page, device=x.device) < first[:, None]
    shifted = cache.view(torch.float8_e4m3fn).float() * power((old - new).clamp(min=-126))[..., None, None]
    again = shifted.to(torch.float8_e4m3fn).view(torch.uint8)
    cache.copy_(torch.where(moved[..., None, None] & before[:, None, :, None], again, cache))
    scale.copy_((new + 127).to(torch.uint8))
    # The new rows; a row without a slot writes back what its place held.
    row = owner.clamp(max=pages - 1)
    y = (x * power(-new)[row][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    spot = torch.where(used, owner * page + off, pages * page)
    flat = torch.cat([cache.transpose(1, 2).reshape(pages * page, heads, dim), cache.new_zeros(1, heads, dim)])
    flat[spot] = y
    cache.copy_(flat[:-1].view(pages, page, heads, dim).transpose(1, 2))


def attend_plain(s):
    k, v, ks, vs = s["cache"]
    page, heads, dim = k.shape[2], k.shape[1], k.shape[3]
    requests, width, longest = s["requests"], s["table"].shape[1], s["longest_query"]
    table = s["table"].clamp(min=0).long()
    seq = s["seq_lens"].long()
    at = torch.arange(width * page, device=k.device)
    inside = (at < seq[:, None])[:, None, :, None]

    def rows(c, sc):  # [requests, heads, tokens, dim]
        x = c[table].view(torch.float8_e4m3fn).float() * power(sc[table].int() - 127)[..., None, None]
        x = x.transpose(1, 2).reshape(requests, heads, width * page, dim)
        return torch.where(inside, x, 0.0)

    keys, values = rows(k, ks), rows(v, vs)
    start = s["query_start"].long()
    new = start[1:] - start[:-1]
    i = torch.arange(longest, device=k.device)
    token = (start[:-1, None] + i).clamp(max=s["tokens"] - 1)
    group = s["q"].shape[1] // heads
    q = s["q"][token].float().view(requests, longest, heads, group, dim).permute(0, 2, 1, 3, 4)
    q = q.reshape(requests, heads, longest * group, dim)
    scores = (torch.matmul(q, keys.transpose(2, 3)) * s["scale"]).view(requests, heads, longest, group, width * page)
    pos = (seq - new)[:, None] + i
    seen = (at <= pos[..., None]) & (at < seq[:, None, None])
    if s["case"]["window"]:
        seen &= at > pos[..., None] - s["case"]["window"]
    seen = seen[:, None, :, None, :]
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(requests, heads, longest * group, -1), values).view(requests, heads, longest, group, dim)
    out = torch.where(total > 0, out / total, 0.0).permute(0, 2, 1, 3, 4).reshape(requests, longest, -1, dim)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(requests, longest, -1)
    # Back to the token axis; rows past the last request's tokens keep what they held.
    t = torch.arange(s["tokens"], device=k.device)
    r = torch.searchsorted(start[1:], t, right=True).clamp(max=requests - 1)
    n = (t - start[r]).clamp(0, longest - 1)
    used = t < start[-1]
    s["out"].copy_(torch.where(used[:, None, None], out[r, n].to(s["out"].dtype), s["out"]))
    s["lse"].copy_(torch.where(used[:, None], lse[r, n], s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    """What run() returns, token by token or request by request in float64; whole numbers have no such value."""
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    if case["op"] == "route":
        return exact_route(case, s)
    if case["op"] == "append":
        return exact_append(s)
    return exact_attend(case, s)


def exact_route(case, s):
    x = s["logits"].double().cpu().numpy()
    tokens, experts = x.shape
    k, groups = case["topk"], case["groups"]
    if case["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + np.exp(-x))
    else:
        score = np.exp(x - x.max(1, keepdims=True))
        score /= score.sum(1, keepdims=True)
    key = x.copy()
    if s["bias"] is not None:  # the selection compares 32-bit sums
        key = (score.astype(np.float32) + s["bias"].cpu().numpy()).astype(np.float64)
    elif groups > 1 and case["group_score"] == 2:
        key = score.copy()
    if groups > 1:
        part = np.sort(key.reshape(tokens, groups, -1), -1)[..., ::-1]
        rank = part[..., 0] if case["group_score"] == 1 else (part[..., 0].astype(np.float32) + part[..., 1].astype(np.float32))
        chosen = np.argsort(-rank, axis=1, kind="stable")[:, : case["group_topk"]]
        allowed = np.zeros((tokens, groups), bool)
        np.put_along_axis(allowed, chosen, True, 1)
        key[~np.repeat(allowed, experts // groups, 1)] = -np.inf
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(score, ids, 1)
    if case["renormalize"]:
        w = w / w.sum(1, keepdims=True)
    return {"ids": None, "weights": w * case["scale"]}


def _round_e4m3(a):
    """Values rounded to the e4m3 grid, halves to even, held at 448."""
    mag = np.abs(a)
    _, e = np.frexp(mag)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.copysign(np.minimum(np.rint(mag / step) * step, 448.0), a)


def exact_append(s):
    out = []
    slots = s["slots"].cpu().numpy()
    page = s["cache"][0].shape[2]
    for x, cache, scale in ((s["k"], s["cache"][0], s["cache"][2]), (s["v"], s["cache"][1], s["cache"][3])):
        x, scale = x.double().cpu().numpy(), scale.cpu().numpy().astype(np.int64) - 127
        values = cache.view(torch.float8_e4m3fn).float().cpu().numpy()
        i = 0
        while i < len(slots):
            n = 1
            while i + n < len(slots) and slots[i + n] == slots[i] + n and slots[i + n] % page:
                n += 1
            if slots[i] >= 0:
                p, off = divmod(int(slots[i]), page)
                rows = x[i:i + n].transpose(1, 0, 2)  # [heads, n, dim]
                amax = np.abs(rows).max((1, 2))
                need = np.where(amax > 0, np.ceil(np.log2(np.maximum(amax, 1e-300) / 448.0)), -127).astype(np.int64)
                need = np.maximum(need, -127)
                now = np.maximum(need, scale[p]) if off else need
                if off:
                    shift = np.ldexp(1.0, scale[p] - now)[:, None, None]
                    values[p, :, :off] = _round_e4m3(values[p, :, :off].astype(np.float64) * shift)
                values[p, :, off:off + n] = _round_e4m3(rows * np.ldexp(1.0, -now)[:, None, None])
                scale[p] = now
            i += n
        out.append(values)
    return {"k": out[0], "v": out[1], "k_scale": None, "v_scale": None}


def exact_attend(case, s):
    page, dim = case["page"], case["head_dim"]
    heads, group = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    out = torch.zeros(s["tokens"], case["q_heads"], dim, dtype=torch.float64, device=DEVICE)
    lse = torch.zeros(s["tokens"], case["q_heads"], dtype=torch.float64, device=DEVICE)
    start, seq, table = s["query_start"].tolist(), s["seq_lens"].tolist(), s["table"].long()
    for r in range(s["requests"]):
        a, b, n = start[r], start[r + 1], seq[r]
        if a == b:
            continue
        pages = table[r, : -(-n // page)]
        q = s["q"][a:b].double().view(b - a, heads, group, dim)
        at = torch.arange(n, device=DEVICE)
        pos = n - (b - a) + torch.arange(b - a, device=DEVICE)[:, None]
        seen = (at <= pos) & (at > pos - (case["window"] or n + 1))
        for h in range(heads):
            k, v = ((c[pages, h].view(torch.float8_e4m3fn).double() * torch.exp2(e[pages, h].double() - 127)[:, None, None])
                    .view(-1, dim)[:n] for c, e in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])))
            logits = torch.einsum("qgd,kd->qgk", q[:, h], k) / math.sqrt(dim)
            logits = logits.masked_fill(~seen[:, None], -math.inf)
            rows = slice(h * group, (h + 1) * group)
            lse[a:b, rows] = torch.logsumexp(logits, -1)
            out[a:b, rows] = torch.softmax(logits, -1) @ v
    return {"out": out, "lse": lse}
