"""What a decode step needs beside its routing, cache and experts: norms, rotary positions, shared pages.

Five operators, each as plain torch arithmetic (``own = False``) and as the
library's call (``own = True``):

* ``norm``: residual addition and root-mean-square norm, with an output in 16
  bits and one in MXFP8 (e4m3 codes, a power-of-two scale for each 32 elements);
* ``rope``: queries and keys rotated by their tokens' positions;
* ``fork``: requests that go on from others' caches: their block tables, and a
  copy of the last page where two would write into it;
* ``reclaim``: the free list of a pool from the tables that hold its pages, and
  (compacting) the pages moved to the pool's front;
* ``shared``: causal attention over the cache of requests in groups, each of
  which shares the pages of a prefix, read once for all of its requests.

The cache is uint8 [pages, kv_heads, page, head_dim] of e4m3 codes for keys and
another for values, with uint8 [pages, kv_heads] E8M0 scales (byte b stands
for 2^(b - 127)).
"""
import math

import torch

own = False

DEVICE = "cuda"
WORKSPACE_BYTES = 32 << 20  # what an attend call may need between its CTAs
LARGEST = {"bytes": 5.5e8, "flops": 6e10}  # the largest listed cases' work


# ------------------------------------------------------------------ the cases
def listed():
    norm = dict(op="norm", hidden=3584, dtype="bfloat16", residual="bfloat16", out=True, codes=True, offset=0.0, pad=0)
    rope = dict(op="rope", q_heads=64, kv_heads=8, head_dim=128, rotary=128, interleaved=False, base=1e6, bands=False,
                factor=1.0, low=1, in_place=False)
    fork = dict(op="fork", page=64, kv_heads=8, head_dim=128, low=1)
    reclaim = dict(op="reclaim", page=64, kv_heads=8, head_dim=128, low=1, done_every=5, group=4, spare=1.0)
    shared = dict(op="shared", page=64, q_heads=64, kv_heads=8, head_dim=128, query=1, prefix_low=1, suffix_low=1,
                  alone_every=0, empty_every=0, pad=0)
    return [
        # The norm in front of the experts for one token: latency alone.
        dict(norm, name="norm_single", tokens=1),
        # A decode batch whose residual stream is held in 32 bits.
        dict(norm, name="norm_batch", tokens=64, residual="float32"),
        # A ragged prompt.
        dict(norm, name="norm_prompt", tokens=16381),
        # The positions of one decode step, far into contexts stretched eightfold.
        dict(rope, name="rope_decode", tokens=64, bands=True, factor=8.0, low=1000, context=131071),
        # Whole prompts, neighbouring elements in pairs, half of each head rotated.
        dict(rope, name="rope_prompt", tokens=12592, interleaved=True, rotary=64, base=1e4, context=1500),
        # Eight prompts that go on in eight samples each, and one layer's pages copied.
        dict(fork, name="fork_samples", parents=8, requests=64, context=8192),
        # A beam step over a large queue with small pages: rows reordered, most pages shared.
        dict(fork, name="fork_beams", parents=1000, requests=1000, context=3000, page=16, kv_heads=4, head_dim=64),
        # The free list after requests have ended, a pool of small pages.
        dict(reclaim, name="reclaim_free", requests=1000, context=3000, page=16, compact=False),
        # A pool that has come apart, moved together, and one layer's pages with it.
        dict(reclaim, name="reclaim_compact", requests=64, context=4096, compact=True),
        # Four samples of one short prompt: latency alone.
        dict(shared, name="shared_samples", requests=4, groups=1, prefix=777, suffix=40),
        # A decode batch under one long instruction text, contexts of their own behind it.
        dict(shared, name="shared_batch", requests=64, groups=1, prefix_low=8192, prefix=8192, suffix=1024),
        # Drafted tokens verified for samples of several prompts, requests without a partner and empty ones between.
        dict(shared, name="shared_groups", requests=48, groups=7, prefix_low=1500, prefix=6000, suffix=400, query=6,
             page=16, q_heads=28, kv_heads=4, head_dim=64, alone_every=5, empty_every=9, pad=3),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    while True:
        case = _draw(rng)
        w = work(case)
        if w["bytes"] <= LARGEST["bytes"] and w["flops"] <= LARGEST["flops"] and state_bytes(case) <= 1.1e10:
            return case


def _draw(rng):
    op = rng.choice(["norm", "rope", "fork", "reclaim", "shared", "shared"])
    if op == "norm":
        hidden = rng.choice([64, 128, 256, 3584, 32 * _log(rng, 1, 512), 8 * _log(rng, 1, 2048), _log(rng, 1, 5000)])
        codes = hidden % 32 == 0 and rng.random() < 0.7
        return dict(op=op, tokens=_log(rng, 1, 16384), hidden=hidden, dtype=rng.choice(["bfloat16", "bfloat16", "float16", "float32"]),
                    residual=rng.choice(["", "bfloat16", "float32"]), out=not codes or rng.random() < 0.7, codes=codes,
                    offset=rng.choice([0.0, 1.0]), pad=rng.choice([0, 0, 8, 5]))
    if op == "rope":
        dim = rng.choice([64, 96, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 3, 4, 8])
        return dict(op=op, tokens=_log(rng, 1, 16384), kv_heads=kv_heads, q_heads=kv_heads * rng.choice([1, 2, 4, 5, 7, 8]),
                    head_dim=dim, rotary=rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)]),
                    interleaved=rng.random() < 0.5, base=rng.choice([1e4, 5e5, 1e6]), bands=rng.random() < 0.5,
                    factor=rng.choice([1.0, 4.0, 8.0, 32.0]), low=1, context=_log(rng, 16, 1 << 20), in_place=rng.random() < 0.3)
    cache = dict(page=rng.choice([16, 32, 64, 128]), kv_heads=rng.choice([1, 2, 3, 4, 8]), head_dim=rng.choice([64, 128, 128, 256]))
    if op == "fork":
        return dict(op=op, parents=_log(rng, 1, 1000), requests=_log(rng, 1, 1000), low=1, context=_log(rng, 1, 16384), **cache)
    if op == "reclaim":
        return dict(op=op, requests=_log(rng, 1, 1024), low=1, context=_log(rng, 1, 16384), done_every=rng.choice([0, 2, 5]),
                    group=rng.choice([1, 4]), spare=rng.choice([0.1, 1.0, 3.0]), compact=rng.random() < 0.5, **cache)
    return dict(op=op, requests=_log(rng, 1, 100), groups=_log(rng, 1, 12), prefix_low=1, prefix=_log(rng, 1, 16384), suffix_low=1,
                suffix=_log(rng, 1, 3000), query=rng.choice([1, 1, rng.randint(2, 9), _log(rng, 2, 300)]),
                q_heads=cache["kv_heads"] * rng.choice([1, 2, 4, 5, 7, 8, 16]), alone_every=rng.choice([0, 4]),
                empty_every=rng.choice([0, 0, 5]), pad=rng.choice([0, 0, 7]), **cache)


# ---------------------------------------------------------------- the lengths
def spread(n, low, high, step):
    """n lengths over [low, high] (low held at most at high), from the numbers alone."""
    low = min(low, high)
    return [low + int(round((high - low) * (((i + 1) * step) % 1.0))) for i in range(n)]


def groups_of(case):
    """Sizes of the groups that the requests come in, one after the other."""
    n = case["requests"]
    groups = min(case["groups"], n)
    ends = [(i + 1) * n // groups for i in range(groups)]
    sizes = [b - a for a, b in zip([0] + ends, ends)]
    if case["alone_every"]:  # some groups come apart into requests of their own
        sizes = [s for i, g in enumerate(sizes) for s in ([1] * g if i % case["alone_every"] == case["alone_every"] - 1 else [g])]
    return sizes


def lengths_of(case):
    """shared: (size, prefix) of each group, then (tokens of the cache, new tokens) of each request, in order."""
    sizes = groups_of(case)
    prefix = spread(len(sizes), case["prefix_low"], case["prefix"], 0.6180339887)
    suffix = spread(case["requests"], case["suffix_low"], case["suffix"], 0.4142135624)
    top = case["query"]
    total, new, r = [], [], 0
    for size, p in zip(sizes, prefix):
        for _ in range(size):
            q = 1 if top == 1 else top // 2 + 1 + int(((r + 1) * 0.7320508076 % 1.0) * (top - top // 2 - 1))
            if case["empty_every"] and r % case["empty_every"] == case["empty_every"] - 1:
                total, new = total + [0], new + [0]
            else:
                total, new = total + [p + max(suffix[r], q)], new + [q]
            r += 1
    return sizes, prefix, total, new


def contexts_of(case):
    """fork, reclaim: the lengths of the rows that hold pages."""
    n = case["parents"] if case["op"] == "fork" else case["requests"]
    lens = spread(n, case["low"], case["context"], 0.6180339887)
    every = case.get("done_every", 0)
    return [0 if every and i % every == every - 1 else c for i, c in enumerate(lens)]


def shares_of(case):
    """reclaim: the pages that the rows of a group share, and the pages held in all."""
    page, lens, shared, held = case["page"], contexts_of(case), [], 0
    for i in range(0, len(lens), case["group"]):
        rows = [c for c in lens[i:i + case["group"]] if c]
        common = min((c // page for c in rows), default=0) // 2 if len(rows) > 1 else 0
        shared.append(common)
        held += sum(-(-c // page) - common for c in rows) + (common if rows else 0)
    return shared, held


def pool_of(case):
    """reclaim: (pages held, pages of the pool)."""
    held = shares_of(case)[1]
    return held, held + 3 + int(held * case["spare"])


def work(case):
    op = case["op"]
    if op == "norm":
        size = {"": 0, "bfloat16": 2, "float16": 2, "float32": 4}
        row = size[case["dtype"]] * (2 if case["out"] else 1) + 2 * size[case["residual"]]
        per = case["hidden"] * row + (case["hidden"] // 32 * 33 if case["codes"] else 0)
        return {"bytes": case["tokens"] * per + 4 * case["hidden"], "flops": 5 * case["tokens"] * case["hidden"]}
    if op == "rope":
        heads, part = case["q_heads"] + case["kv_heads"], case["rotary"] if case["in_place"] else case["head_dim"]
        return {"bytes": case["tokens"] * (4 * heads * part + 4), "flops": 3 * case["tokens"] * heads * case["rotary"]}
    row = 2 * case["kv_heads"] * case["head_dim"]  # bytes of a token's keys and values
    if op == "fork":
        lens, page = contexts_of(case), case["page"]
        table = moved = 0
        seen = set()
        for p in parents_of(case):
            table += -(-lens[p] // page)
            moved += lens[p] % page if p in seen else 0
            seen.add(p)
        width = max(-(-c // page) for c in lens) + 1
        return {"bytes": 4 * table + 4 * case["requests"] * (width + 6) + 2 * row * moved, "flops": 0}
    if op == "reclaim":
        held, pages = pool_of(case)
        entries = sum(-(-c // case["page"]) for c in contexts_of(case))
        moves = held * (1 - held / pages)  # on the average
        out = 4 * entries + moves * (12 + 2 * row * case["page"]) if case["compact"] else 0
        return {"bytes": 4 * entries + 4 * (pages - held) + out, "flops": 0}
    sizes, prefix, total, new = lengths_of(case)
    seen, pairs, r = 0, 0, 0
    for size, p in zip(sizes, prefix):
        live = [(c, q) for c, q in zip(total[r:r + size], new[r:r + size]) if q]
        seen += (p if live else 0) + sum(c - p for c, q in live)
        pairs += sum(q * (c - q) + q * (q + 1) // 2 for c, q in live)
        r += size
    out = sum(new) * case["q_heads"] * (case["head_dim"] * 4 + 4)
    return {"bytes": row * seen + 2 * (seen // case["page"]) * case["kv_heads"] + out,
            "flops": 4 * pairs * case["q_heads"] * case["head_dim"]}


def state_bytes(case):
    """About what a case's inputs and its plain form hold at once."""
    op = case["op"]
    if op == "norm":
        return 40 * case["tokens"] * case["hidden"]
    if op == "rope":
        return 24 * case["tokens"] * (case["q_heads"] + case["kv_heads"]) * case["head_dim"]
    page = 2 * case["page"] * case["kv_heads"] * case["head_dim"]
    if op == "fork":
        lens = contexts_of(case)
        return page * (sum(-(-c // case["page"]) for c in lens) + 4 * case["requests"])
    if op == "reclaim":
        return 16 * case["requests"] * case["context"] + (3 * page * pool_of(case)[1] if case["compact"] else 0)
    sizes, prefix, total, new = lengths_of(case)
    longest = max(total) + 2 * case["page"]
    return 4 * case["requests"] * longest * (4 * case["kv_heads"] * case["head_dim"] + 4 * max(new + [1]) * case["q_heads"])


def parents_of(case):
    """fork: the row that each request goes on from: samples by turns, beams with some rows taken twice and some dropped."""
    n, p = case["requests"], case["parents"]
    return [int(((i * 0.3819660113) % 1.0) * p) if n <= p else i * p // n for i in range(n)]


# ----------------------------------------------------------------- the inputs
def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEVICE)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    s = dict(case=dict(case))
    {"norm": prepare_norm, "rope": prepare_rope, "fork": prepare_fork, "reclaim": prepare_reclaim,
     "shared": prepare_shared}[case["op"]](case, s, g, seed)
    return s


def prepare_norm(case, s, g, seed):
    t, n = case["tokens"], case["hidden"]
    dtype = getattr(torch, case["dtype"])
    # Rows of a product's output, some channels of the residual stream far larger than the others.
    x = torch.randn(t, n + case["pad"], generator=g, device=DEVICE)
    s["x"] = x.to(dtype)[:, :n]
    s["residual"] = s["residual_out"] = None
    if case["residual"]:
        loud = 1 + 40 * (torch.rand(n, generator=g, device=DEVICE) > 0.995)
        s["residual"] = (3 * torch.randn(t, n, generator=g, device=DEVICE) * loud).to(getattr(torch, case["residual"]))
        s["residual_out"] = torch.empty_like(s["residual"])
    s["weight"] = (1 - case["offset"] + 0.2 * torch.randn(n, generator=g, device=DEVICE)).contiguous()
    s["out"] = torch.empty(t, n, dtype=dtype, device=DEVICE) if case["out"] else None
    s["codes"] = torch.empty(t, n, dtype=torch.uint8, device=DEVICE) if case["codes"] else None
    s["scales"] = torch.empty(t, n // 32, dtype=torch.uint8, device=DEVICE) if case["codes"] else None


def frequencies(case):
    """Radians a position of each pair of dimensions; `bands`: long waves slowed by the factor, short ones kept, a ramp between."""
    n = case["rotary"]
    out = []
    for i in range(n // 2):
        f = case["base"] ** (-2.0 * i / n)
        if case["bands"]:
            turns = 8192 * f / math.tau  # over the length that the model was trained with
            keep = min(max((turns - 1.0) / (4.0 - 1.0), 0.0), 1.0)
            f = f * keep + f / case["factor"] * (1 - keep)
        else:
            f = f / case["factor"]
        out.append(f)
    return out


def prepare_rope(case, s, g, seed):
    t, dim, heads = case["tokens"], case["head_dim"], case["q_heads"] + case["kv_heads"]
    f = frequencies(case)
    s["frequencies"] = torch.tensor(f, dtype=torch.float64, device=DEVICE)
    # The library's table holds them in units of 2^-64 turns.
    turns = [round(v / math.tau * 2.0 ** 64) for v in f]
    s["turns"] = ints([v - (1 << 64) if v >= 1 << 63 else v for v in turns], torch.int64)
    # One projection gives queries, keys and values side by side.
    qkv = torch.randn(t, heads + case["kv_heads"], dim, generator=g, device=DEVICE).to(torch.bfloat16)
    s["q"], s["k"] = qkv[:, :case["q_heads"]], qkv[:, case["q_heads"]:heads]
    if case["in_place"]:
        s["q_out"], s["k_out"] = s["q"], s["k"]
    else:
        s["q_out"] = torch.empty(t, case["q_heads"], dim, dtype=torch.bfloat16, device=DEVICE)
        s["k_out"] = torch.empty(t, case["kv_heads"], dim, dtype=torch.bfloat16, device=DEVICE)
    low = min(case["low"], case["context"])
    first = torch.randint(low, case["context"] + 1, (1 + t // 700,), generator=g, device=DEVICE)
    at = torch.arange(t, device=DEVICE)
    if t <= 700:  # tokens of as many requests
        s["positions"] = torch.randint(low, case["context"] + 1, (t,), generator=g, device=DEVICE).int()
    else:  # chunks of prompts
        s["positions"] = ((first[at // 700] + at % 700) % case["context"]).int()


def codes(pool, heads, page, dim, g):
    """e4m3 codes as a cache of unit normals has them, with scales that differ by page and head."""
    data = torch.empty(pool, heads, page, dim, dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 26) // (heads * page * dim))
    for i in range(0, pool, step):
        part = torch.randn(data[i:i + step].shape, generator=g, device=DEVICE)
        data[i:i + step] = (part * 90).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return data, torch.randint(119, 122, (pool, heads), generator=g, device=DEVICE, dtype=torch.uint8)


def cache_of(case, pages, g):
    """k, v, k_scale, v_scale; one page more than the tables and the free list know."""
    k, v = (codes(pages + 1, case["kv_heads"], case["page"], case["head_dim"], g) for _ in range(2))
    return k[0], v[0], k[1], v[1]


def table_of(needed, width, ids):
    """Rows of `needed` pages each out of ids, one after the other; -1 behind them."""
    n = ints(needed, torch.int64)
    at = torch.arange(width, device=DEVICE)
    start = torch.cumsum(n, 0) - n
    return torch.where(at < n[:, None], ids[(start[:, None] + at).clamp(max=ids.numel() - 1)], -1).int().contiguous()


def prepare_fork(case, s, g, seed):
    lens, page, requests = contexts_of(case), case["page"], case["requests"]
    needed = [-(-c // page) for c in lens]
    held, width = sum(needed), max(needed) + 1
    pages = held + requests + 3
    ids = torch.randperm(pages, generator=g, device=DEVICE).int()
    order = torch.randperm(requests, generator=torch.Generator().manual_seed(seed)).tolist()
    parents = parents_of(case)
    s.update(parents=ints([parents[i] for i in order]), seq_lens=ints(lens), table=table_of(needed, width, ids), page=page,
             free=ids[held:].contiguous(), free_head=ints([0]), cache=cache_of(case, pages, g),
             out_table=torch.empty(requests, width, dtype=torch.int32, device=DEVICE),
             out_lens=torch.empty(requests, dtype=torch.int32, device=DEVICE),
             moves=torch.empty(requests, 3, dtype=torch.int32, device=DEVICE),
             counts=torch.empty(4, dtype=torch.int32, device=DEVICE))


def prepare_reclaim(case, s, g, seed):
    lens, page = contexts_of(case), case["page"]
    shared, held = shares_of(case)
    pages = pool_of(case)[1]
    needed = [-(-c // page) for c in lens]
    width = max(needed + [1]) + 1
    ids = torch.randperm(pages, generator=g, device=DEVICE).int()
    table = torch.full((len(lens), width), -1, dtype=torch.int64)
    at, first, host = 0, 0, ids.cpu().long()
    for i, n in enumerate(needed):
        if i % case["group"] == 0:
            first = at  # the group's common pages
            at += shared[i // case["group"]] if any(needed[i:i + case["group"]]) else 0
        common = shared[i // case["group"]] if n else 0
        table[i, :common] = host[first:first + common]
        table[i, common:n] = host[at:at + n - common]
        at += n - common
        if not n:  # a request that has ended: its row still holds what it held
            table[i] = torch.randint(0, pages, (width,), generator=torch.Generator().manual_seed(seed + i))
    s.update(seq_lens=ints(lens), table=table.to(DEVICE).int().contiguous(), page=page, pages=pages,
             free=torch.zeros(pages, dtype=torch.int32, device=DEVICE), counts=torch.empty(4, dtype=torch.int32, device=DEVICE),
             workspace=torch.zeros(1024 + 8 * pages, dtype=torch.uint8, device=DEVICE), out_table=None, moves=None)
    if case["compact"]:
        s["out_table"] = torch.empty_like(s["table"])
        s["moves"] = torch.zeros(max(1, pages // 2), 3, dtype=torch.int32, device=DEVICE)
        s["cache"] = cache_of(case, pages, g)


def prepare_shared(case, s, g, seed):
    sizes, prefix, total, new = lengths_of(case)
    page, dim, tokens, requests = case["page"], case["head_dim"], sum(new) + case["pad"], len(new)
    needed, common, r = [-(-c // page) for c in total], [], 0
    for size, p in zip(sizes, prefix):
        common += [p // page if size > 1 else 0] * size
    width = max(needed + [1]) + 1
    own_pages = sum(max(n - c, 0) for n, c in zip(needed, common))
    pages = own_pages + sum(p // page for p in prefix) + 1
    ids = torch.randperm(pages, generator=g, device=DEVICE).int()
    host, table, at = ids.cpu().long(), torch.full((requests, width), -1, dtype=torch.int64), 0
    for size, p in zip(sizes, prefix):
        first, at = at, at + (p // page if size > 1 else 0)
        for i in range(r, r + size):
            c = min(common[i], needed[i])
            table[i, :c] = host[first:first + c]
            table[i, c:needed[i]] = host[at:at + needed[i] - c]
            at += needed[i] - c
        r += size
    start = [0]
    for q in new:
        start.append(start[-1] + q)
    ends = [0]
    for size in sizes:
        ends.append(ends[-1] + size)
    s.update(table=table.to(DEVICE).int().contiguous(), query_start=ints(start), seq_lens=ints(total), group_start=ints(ends),
             prefix_lens=ints(prefix), tokens=tokens, requests=requests, longest_query=max(new + [1]), scale=1.0 / math.sqrt(dim))
    s["cache"] = cache_of(case, pages, g)
    s["q"] = torch.randn(tokens, case["q_heads"], dim, generator=g, device=DEVICE).to(torch.bfloat16)
    s["out"] = torch.zeros(tokens, case["q_heads"], dim, dtype=torch.bfloat16, device=DEVICE)
    s["lse"] = torch.zeros(tokens, case["q_heads"], dtype=torch.float32, device=DEVICE)
    s["workspace"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device=DEVICE)
    s["scratch"] = torch.zeros(65536 + 4 * tokens * case["q_heads"] * (dim + 2), dtype=torch.uint8, device=DEVICE)


# ------------------------------------------------------------ one pass through
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": norm_own, "rope": rope_own, "fork": fork_own, "reclaim": reclaim_own, "shared": shared_own}[op](state)
    return {"norm": norm_plain, "rope": rope_plain, "fork": fork_plain, "reclaim": reclaim_plain, "shared": shared_plain}[op](state)


def norm_own(s):
    import mxfp4_weight_mxfp8_gb300 as moe

    moe.moe_norm(s["x"], s["weight"], s["out"], residual=s["residual"], residual_out=s["residual_out"], codes=s["codes"],
                 scales=s["scales"], eps=1e-6, weight_offset=s["case"]["offset"])
    return norm_outputs(s)


def rope_own(s):
    import mxfp4_weight_mxfp8_gb300 as moe

    moe.moe_rope(s["positions"], s["turns"], s["q"], s["k"], s["q_out"], s["k_out"], interleaved=s["case"]["interleaved"])
    return {"q": s["q_out"], "k": s["k_out"]}


def fork_own(s):
    import mxfp4_weight_mxfp8_gb300 as moe

    moe.moe_kv_fork(s["parents"], s["table"], s["seq_lens"], s["page"], s["free"], s["free_head"], s["out_table"],
                    s["out_lens"], s["moves"], s["counts"])
    moe.moe_kv_copy(s["cache"], s["moves"])
    return fork_outputs(s)


def reclaim_own(s):
    import mxfp4_weight_mxfp8_gb300 as moe

    moe.moe_kv_reclaim(s["table"], s["seq_lens"], s["page"], s["free"], s["counts"], s["workspace"],
                       out_table=s["out_table"], moves=s["moves"])
    if s["case"]["compact"]:
        moe.moe_kv_copy(s["cache"], s["moves"], s["counts"][2:3])
    return reclaim_outputs(s)


def shared_own(s):
    import mxfp4_weight_mxfp8_gb300 as moe

    moe.moe_kv_attend_shared(s["cache"], s["q"], s["table"], s["query_start"], s["seq_lens"], s["group_start"],
                             s["prefix_lens"], s["out"], s["workspace"], s["scratch"], lse=s["lse"], scale=s["scale"])
    return {"out": s["out"], "lse": s["lse"]}


def norm_outputs(s):
    """Codes and scales as the numbers that they stand for."""
    both = s["codes"] is not None
    return {"out": s["out"], "residual": s["residual_out"], "codes": s["codes"].view(torch.float8_e4m3fn) if both else None,
            "scales": s["scales"].view(torch.float8_e8m0fnu) if both else None}


def cache_values(cache):
    """The cache as the numbers that its codes stand for, next to their exponents."""
    k, v, ks, vs = cache
    return {"k": k.view(torch.float8_e4m3fn), "v": v.view(torch.float8_e4m3fn), "k_scale": ks, "v_scale": vs}


def fork_outputs(s):
    return {"table": s["out_table"], "lens": s["out_lens"], "moves": s["moves"], "counts": s["counts"], **cache_values(s["cache"])}


def reclaim_outputs(s):
    out = {"free": s["free"], "counts": s["counts"]}
    if s["case"]["compact"]:
        out.update(table=s["out_table"], moves=s["moves"], **cache_values(s["cache"]))
    return out


# -------------------------------------------------------------- the plain form
def power(e):
    """2^e in 32 bits, exactly, for whole e in [-127, 127]."""
    e = e.int()
    return torch.where(e > -127, (e + 127) << 23, 0x00400000).view(torch.float32)


def exponent(amax):
    """The smallest E with amax <= 448 * 2^E, at least -127; -127 for zero and what 32 bits hold without a leading one."""
    m, e = torch.frexp(amax)
    return torch.where(amax >= 2.0 ** -126, e - 9 + (m > 0.875).int(), -127).clamp(-127, 127).int()


def norm_plain(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
        s["residual_out"].copy_(h)
    mean = (h * h).sum(-1, keepdim=True) / h.shape[-1]
    y = h * (1.0 / torch.sqrt(mean + 1e-6)) * (s["weight"] + s["case"]["offset"])
    if s["out"] is not None:
        s["out"].copy_(y)
    if s["codes"] is not None:
        b = y.view(y.shape[0], -1, 32)
        e = exponent(b.abs().amax(-1))
        s["codes"].copy_((b * power(-e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view_as(y))
        s["scales"].copy_((e + 127).to(torch.uint8))
    return norm_outputs(s)


def rope_plain(s):
    angle = s["positions"].double()[:, None] * s["frequencies"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    n = s["case"]["rotary"]
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        f = x[..., :n].float()
        if s["case"]["interleaved"]:
            a, b = f[..., 0::2], f[..., 1::2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = f[..., : n // 2], f[..., n // 2:]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        out[..., n:] = x[..., n:]
        out[..., :n] = turned.to(out.dtype)
    return {"q": s["q_out"], "k": s["k_out"]}


def fork_plain(s):
    page, width, requests = s["page"], s["table"].shape[1], s["parents"].numel()
    parent = s["parents"].long()
    lens = s["seq_lens"].long()[parent]
    at, r = torch.arange(width, device=lens.device), torch.arange(requests, device=lens.device)
    needed = (lens + page - 1) // page
    table = torch.where(at < needed[:, None], s["table"][parent], -1)
    # The first request that goes on from a row keeps its last page; the others take a copy, where it is not full.
    first = torch.full((s["table"].shape[0],), requests, device=lens.device).scatter_reduce_(0, parent, r, "amin")
    rest = lens % page
    last = (needed - 1).clamp(min=0)
    entry = table.gather(1, last[:, None])[:, 0].long()
    wants = (first[parent] != r) & (rest > 0) & (entry >= 0)
    rank = s["free_head"].long() + torch.cumsum(wants, 0) - wants.long()
    free = s["free"].numel()
    fresh = torch.where(rank < free, s["free"][rank.clamp(0, free - 1)], -1)
    table = torch.where(wants[:, None] & (at == last[:, None]), fresh[:, None], table)
    moved = wants & (fresh >= 0)
    none = torch.full_like(entry, -1)
    s["moves"].copy_(torch.stack((torch.where(moved, entry, none), torch.where(moved, fresh.long(), none), torch.where(moved, rest, 0)), 1))
    s["out_table"].copy_(table)
    s["out_lens"].copy_(lens)
    taken = wants.sum()
    s["counts"].copy_(torch.stack((moved.sum(), s["free_head"][0].long() + taken, lens.max(), 8 * (s["free_head"][0] + taken > free).long())))
    copy_plain(s["cache"], s["moves"])
    return fork_outputs(s)


def copy_plain(cache, moves, count=None):
    """Rows [0, tokens) of page `from` into page `to`; moves that are none go from the cache's spare page into itself."""
    spare, page = cache[0].shape[0] - 1, cache[0].shape[2]
    source, to, tokens = moves.long().unbind(1)
    used = to >= 0
    if count is not None:
        used &= torch.arange(to.numel(), device=to.device) < count
    source, to, tokens = torch.where(used, source, spare), torch.where(used, to, spare), torch.where(used, tokens, page)
    kept = (torch.arange(page, device=to.device) < tokens[:, None])[:, None, :, None]
    for c in cache[:2]:
        c[to] = torch.where(kept, c[source], c[to])
    for c in cache[2:]:
        c[to] = c[source]


def reclaim_plain(s):
    page, pages, width = s["page"], s["pages"], s["table"].shape[1]
    lens = s["seq_lens"].long()
    needed = (lens + page - 1) // page
    inside = torch.arange(width, device=lens.device) < needed[:, None]
    entries = torch.where(inside, s["table"].long(), pages)
    held = torch.zeros(pages + 1, dtype=torch.bool, device=lens.device)
    held[entries.flatten()] = True
    held = held[:-1]
    count, at = held.sum(), torch.arange(pages, device=lens.device)
    if not s["case"]["compact"]:
        # Free pages in rising order at the list's end, so that its last one is the pool's.
        rank = torch.cumsum(~held, 0) - 1
        spot = torch.where(held, pages, count + rank)
        s["free"].copy_(torch.cat((s["free"], s["free"][:1])).scatter(0, spot, at.int())[:-1])
        s["counts"].copy_(torch.stack((count, count, count * 0, count * 0)))
        return reclaim_outputs(s)
    # Held pages from `count` on go to the free places before it, both in rising order.
    leaves, place = held & (at >= count), ~held & (at < count)
    moves = leaves.sum()
    leaving, placing = torch.cumsum(leaves, 0) - 1, torch.cumsum(place, 0) - 1
    source = torch.full((pages + 1,), -1, device=lens.device).scatter(0, torch.where(leaves, leaving, pages), at)
    target = torch.full((pages + 1,), -1, device=lens.device).scatter(0, torch.where(place, placing, pages), at)
    to = torch.where(leaves, target[leaving.clamp(min=0)], at)
    n = s["moves"].shape[0]
    listed_moves = torch.stack((source[:n], target[:n], torch.full_like(source[:n], page)), 1)
    s["moves"].copy_(torch.where(torch.arange(n, device=lens.device)[:, None] < moves, listed_moves, s["moves"]))
    s["out_table"].copy_(torch.where(inside, to[entries.clamp(max=pages - 1)], -1))
    s["free"].copy_(torch.where(at >= count, at, s["free"].long()))
    s["counts"].copy_(torch.stack((count, count, moves, moves * 0)))
    copy_plain(s["cache"], s["moves"], moves)
    return reclaim_outputs(s)


def shared_plain(s):
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
    seen = ((at <= pos[..., None]) & (at < seq[:, None, None]))[:, None, :, None, :]
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
    """What run() returns, from the definition in float64; whole numbers and what is only moved have no such value."""
    if case["op"] in ("fork", "reclaim"):
        return None
    s = prepare(case, seed)
    return {"norm": exact_norm, "rope": exact_rope, "shared": exact_shared}[case["op"]](case, s)


def exact_norm(case, s):
    h = s["x"].double()
    if s["residual"] is not None:
        h = h + s["residual"].double()
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + 1e-6) * (s["weight"].double() + case["offset"])
    found = {"out": y if case["out"] else None, "residual": h if case["residual"] else None, "codes": None, "scales": None}
    if case["codes"]:
        blocks = y.view(y.shape[0], -1, 32)
        e = torch.ceil(torch.log2(blocks.abs().amax(-1).clamp(min=1e-300) / 448.0)).clamp(-127, 127)
        v = blocks * torch.exp2(-e)[..., None]
        # To the nearest of 3 places after the leading one, halves to even.
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        found["codes"] = (torch.round(v / step) * step).clamp(-448, 448).view_as(y)
        found["scales"] = torch.exp2(e)
    return found


def exact_rope(case, s):
    out = {}
    pairs = case["rotary"] // 2
    angle = s["positions"].double()[:, None] * torch.tensor(frequencies(case), dtype=torch.float64, device=DEVICE)
    unit = torch.polar(torch.ones_like(angle), angle)[:, None]
    for name in ("q", "k"):
        x = s[name].double()
        y = x.clone()
        i = torch.arange(pairs, device=DEVICE)
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + pairs)
        z = torch.complex(x[..., first], x[..., second]) * unit
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    return out


def exact_shared(case, s):
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
        pos = n - (b - a) + torch.arange(b - a, device=DEVICE)[:, None]
        seen = torch.arange(n, device=DEVICE) <= pos
        k, v = ((c[pages].view(torch.float8_e4m3fn).double() * torch.exp2(e[pages].double() - 127)[:, :, None, None])
                .transpose(0, 1).reshape(heads, -1, dim)[:, :n] for c, e in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])))
        logits = torch.einsum("qhgd,hkd->qhgk", q, k) / math.sqrt(dim)
        logits = logits.masked_fill(~seen[:, None, None], -math.inf)
        lse[a:b] = torch.logsumexp(logits, -1).view(b - a, -1)
        out[a:b] = torch.einsum("qhgk,hkd->qhgd", torch.softmax(logits, -1), v).reshape(b - a, -1, dim)
    return {"out": out, "lse": lse}
