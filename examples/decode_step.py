"""A decoder layer's decode step on the library's operators, from a prompt on.

For each step: plan the new tokens' pages and slots, norm and project, rotate
queries and keys by their positions, write keys and values into the 8-bit cache,
attend over it, add and norm, route, and run the top-16 experts with their
routing weights. With --samples, every prompt goes on in several samples, which
share its pages; at the end the samples but the first end, and the pool is
compacted. Random weights; the projections are plain matrix products.

    python examples/decode_step.py [--steps N] [--requests R] [--prompt TOKENS] [--samples S]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_weight_mxfp8_gb300 as moe  # noqa: E402
import workload  # noqa: E402


class DecoderLayer:
    """Attention over the paged cache, then the routed experts; both with a residual."""

    def __init__(self, experts: int, hidden: int, inter: int, q_heads: int, kv_heads: int, head_dim: int, pages: int,
                 page_tokens: int, seed: int = 0):
        g = torch.Generator().manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g) * cols ** -0.5).to(torch.bfloat16).cuda()

        self.q_heads, self.kv_heads, self.dim = q_heads, kv_heads, head_dim
        self.qkv = weight((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.o = weight(hidden, q_heads * head_dim)
        self.gate = weight(experts, hidden)
        self.norms = torch.ones(2, hidden, device="cuda")
        self.turns = moe.moe_rope_turns(head_dim, device="cuda")
        self.bias = torch.zeros(experts, device="cuda")
        weights = workload.make_weights(experts, hidden, inter, seed13=seed, seed2=seed + 1)
        self.experts = moe.MoeLayer(tuple(torch.from_numpy(w).cuda() for w in weights))
        self.cache = moe.KvCache(pages, kv_heads, page_tokens, head_dim)

    def __call__(self, x, step):
        tokens = x.shape[0]
        h, residual = torch.empty_like(x), torch.empty_like(x)
        moe.moe_norm(x, self.norms[0], h)
        qkv = (h @ self.qkv.t()).view(tokens, -1, self.dim)
        q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)  # strided views: read in place
        moe.moe_rope(step.positions, self.turns, q, k)  # in place
        self.cache.append(k, v, step.slots)
        if step.group_start is None:
            attended = self.cache.attend(q, step.block_table, step.query_start, step.seq_lens)
        else:
            attended = self.cache.attend_shared(q, step.block_table, step.query_start, step.seq_lens, step.group_start,
                                                step.prefix_lens)
        moe.moe_norm(attended.view(tokens, -1) @ self.o.t(), self.norms[1], h, residual=x, residual_out=residual)
        ids = torch.empty(tokens, moe.TOPK, dtype=torch.int32, device=x.device)
        weights = torch.empty(tokens, moe.TOPK, device=x.device)
        moe.moe_route(h @ self.gate.t(), ids, weights, scoring=moe.SCORE_SIGMOID, bias=self.bias)
        out = torch.empty_like(x)
        for at in range(0, tokens, moe.MAX_BATCH):  # the layer takes up to 256 tokens a call
            rows = slice(at, min(at + moe.MAX_BATCH, tokens))
            moe.moe_run_combined(self.experts.handle, h[rows], ids[rows], weights[rows], out[rows],
                                 rows.stop - rows.start)
        return residual + out


class Requests:
    """The requests' block table and lengths; plan() makes room for each one's new tokens, on the device."""

    def __init__(self, requests: int, width: int, pages: int, page_tokens: int):
        def ints(*shape):
            return torch.zeros(*shape, dtype=torch.int32, device="cuda")

        self.page_tokens = page_tokens
        self.block_table = ints(requests, width) - 1
        self.query_start, self.seq_lens = ints(requests + 1), ints(requests)
        self.free, self.head = torch.arange(pages, dtype=torch.int32, device="cuda"), ints(1)
        self.counts = ints(4)
        self.group_start = self.prefix_lens = None  # of requests that share a prefix

    def fork(self, samples: int, caches):
        """Every request goes on in `samples` of its own, one after the other; their prompts' pages are shared."""
        requests, width = self.block_table.shape
        parents = torch.arange(requests, dtype=torch.int32, device="cuda").repeat_interleave(samples)
        table = torch.empty(requests * samples, width, dtype=torch.int32, device="cuda")
        lens, moves = torch.empty_like(parents), torch.empty(requests * samples, 3, dtype=torch.int32, device="cuda")
        counts = torch.empty_like(self.counts)
        moe.moe_kv_fork(parents, self.block_table, self.seq_lens, self.page_tokens, self.free, self.head, table, lens, moves, counts)
        for cache in caches:  # each layer's
            cache.copy(moves)
        self.group_start = torch.arange(0, requests * samples + 1, samples, dtype=torch.int32, device="cuda")
        self.prefix_lens, self.seq_lens, self.block_table = self.seq_lens, lens, table
        self.query_start = torch.zeros(requests * samples + 1, dtype=torch.int32, device="cuda")
        self.counts, self.head = counts, counts[1:2]

    def end(self, ended, caches):
        """The requests whose numbers are in `ended` end; the pages still held move to the pool's front."""
        self.seq_lens[ended] = 0
        pages = self.free.numel()
        moves = torch.empty(max(1, pages // 2), 3, dtype=torch.int32, device="cuda")
        self.counts = torch.empty_like(self.counts)
        moe.moe_kv_reclaim(self.block_table, self.seq_lens, self.page_tokens, self.free, self.counts,
                           torch.empty(moe.moe_kv_reclaim_bytes(pages), dtype=torch.uint8, device="cuda"), self.block_table, moves)
        for cache in caches:
            cache.copy(moves, self.counts[2:3])
        self.head = self.counts[1:2]

    def plan(self, query_lens, tokens: int):
        context = self.seq_lens.clone()
        self.positions = torch.empty(tokens, dtype=torch.int32, device="cuda")
        self.slots = torch.empty(tokens, dtype=torch.int64, device="cuda")
        self.counts = torch.empty_like(self.counts)  # the last one still holds the free list's head
        moe.moe_kv_plan(context, query_lens, self.page_tokens, self.block_table, self.free, self.head, self.query_start,
                        self.seq_lens, self.positions, self.slots, self.counts)
        self.head = self.counts[1:2]
        return self


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--prompt", type=int, default=37)
    ap.add_argument("--samples", type=int, default=1)
    a = ap.parse_args(argv)
    page, pages = 16, a.requests * a.samples * ((a.prompt + a.steps) // 16 + 2)
    layer = DecoderLayer(experts=32, hidden=256, inter=64, q_heads=8, kv_heads=2, head_dim=64, pages=pages, page_tokens=page)
    step = Requests(a.requests, (a.prompt + a.steps) // page + 2, pages, page)
    g = torch.Generator().manual_seed(1)
    lens = torch.tensor([a.prompt - r % a.prompt for r in range(a.requests)], dtype=torch.int32)
    x = torch.randn(int(lens.sum()), 256, generator=g).to(torch.bfloat16).cuda()
    y = layer(x, step.plan(lens.cuda(), x.shape[0]))
    print(f"prompts: {x.shape[0]} tokens")
    x = y[step.query_start[1:].long() - 1]  # each request's last row goes on
    errors = step.counts[3:4].clone()
    if a.samples > 1:
        step.fork(a.samples, [layer.cache])
        errors += step.counts[3:4]
        x = x.repeat_interleave(a.samples, 0)
        x = x + 0.1 * torch.randn(x.shape, generator=g).to(torch.bfloat16).cuda()  # the samples go different ways
    ones = torch.ones(a.requests * a.samples, dtype=torch.int32, device="cuda")
    for i in range(a.steps):
        x = y = layer(x, step.plan(ones, a.requests * a.samples))
        errors += step.counts[3:4]
        print(f"step {i}: lengths {step.seq_lens.tolist()}, pages taken {step.head.item()}, |y| {y.float().norm():.4f}")
    if a.samples > 1:
        step.end([r for r in range(a.requests * a.samples) if r % a.samples], [layer.cache])
        errors += step.counts[3:4]
        print(f"samples ended: {step.counts[0].item()} pages held, {step.counts[2].item()} moved to the front")
    if (moe.moe_sync_status(layer.experts.handle) != moe.MOE_OK or layer.cache.status() != moe.MOE_OK
            or errors.item() != 0):
        raise SystemExit("the device reported an error")
    layer.experts.close()
    return y


if __name__ == "__main__":
    main()
