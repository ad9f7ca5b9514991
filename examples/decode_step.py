"""A decoder layer's decode step on the library's operators, from a prompt on.

For each step: plan the new tokens' pages and slots, project, write keys and
values into the 8-bit cache, attend over it, route, and run the top-16
experts with their routing weights. Random weights; the projections are plain
matrix products.

    python examples/decode_step.py [--steps N] [--requests R] [--prompt TOKENS]
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
        self.bias = torch.zeros(experts, device="cuda")
        weights = workload.make_weights(experts, hidden, inter, seed13=seed, seed2=seed + 1)
        self.experts = moe.MoeLayer(tuple(torch.from_numpy(w).cuda() for w in weights))
        self.cache = moe.KvCache(pages, kv_heads, page_tokens, head_dim)

    def __call__(self, x, step):
        tokens = x.shape[0]
        qkv = (norm(x) @ self.qkv.t()).view(tokens, -1, self.dim)
        q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)  # strided views: read in place
        self.cache.append(k, v, step.slots)
        attended = self.cache.attend(q, step.block_table, step.query_start, step.seq_lens)
        x = x + attended.view(tokens, -1) @ self.o.t()
        h = norm(x)
        ids = torch.empty(tokens, moe.TOPK, dtype=torch.int32, device=x.device)
        weights = torch.empty(tokens, moe.TOPK, device=x.device)
        moe.moe_route(h @ self.gate.t(), ids, weights, scoring=moe.SCORE_SIGMOID, bias=self.bias)
        out = torch.empty_like(x)
        for at in range(0, tokens, moe.MAX_BATCH):  # the layer takes up to 256 tokens a call
            rows = slice(at, min(at + moe.MAX_BATCH, tokens))
            moe.moe_run_combined(self.experts.handle, h[rows], ids[rows], weights[rows], out[rows],
                                 rows.stop - rows.start)
        return x + out


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

    def plan(self, query_lens, tokens: int):
        context = self.seq_lens.clone()
        self.positions = torch.empty(tokens, dtype=torch.int32, device="cuda")
        self.slots = torch.empty(tokens, dtype=torch.int64, device="cuda")
        self.counts = torch.empty_like(self.counts)  # the last one still holds the free list's head
        moe.moe_kv_plan(context, query_lens, self.page_tokens, self.block_table, self.free, self.head, self.query_start,
                        self.seq_lens, self.positions, self.slots, self.counts)
        self.head = self.counts[1:2]
        return self


def norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--prompt", type=int, default=37)
    a = ap.parse_args(argv)
    page, pages = 16, a.requests * ((a.prompt + a.steps) // 16 + 2)
    layer = DecoderLayer(experts=32, hidden=256, inter=64, q_heads=8, kv_heads=2, head_dim=64, pages=pages, page_tokens=page)
    step = Requests(a.requests, (a.prompt + a.steps) // page + 2, pages, page)
    g = torch.Generator().manual_seed(1)
    lens = torch.tensor([a.prompt - r % a.prompt for r in range(a.requests)], dtype=torch.int32)
    x = torch.randn(int(lens.sum()), 256, generator=g).to(torch.bfloat16).cuda()
    y = layer(x, step.plan(lens.cuda(), x.shape[0]))
    print(f"prompts: {x.shape[0]} tokens")
    ones = torch.ones(a.requests, dtype=torch.int32, device="cuda")
    for i in range(a.steps):
        x = y[step.query_start[1:].long() - 1]  # each request's last row goes on
        y = layer(x, step.plan(ones, a.requests))
        print(f"step {i}: lengths {step.seq_lens.tolist()}, pages taken {step.head.item()}, |y| {y.float().norm():.4f}")
    if (moe.moe_sync_status(layer.experts.handle) != moe.MOE_OK or layer.cache.status() != moe.MOE_OK
            or step.counts[3].item() != 0):
        raise SystemExit("the device reported an error")
    layer.experts.close()
    return y


if __name__ == "__main__":
    main()
