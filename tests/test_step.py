"""The operators of a step one after the other, as a layer uses them; a captured step; the example with samples."""
from __future__ import annotations

import importlib.util
import math
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__

    __graft_entry__.build()
    import mxfp4_weight_mxfp8_gb300 as moe

    return moe


def example():
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
def test_norm_rope_append_attend_against_the_formula(moe):
    """One layer's attention part for two requests with earlier tokens, in 64 bits from the same inputs.

    The 8-bit cache bounds the agreement: a key or value of the cache is within 2^-4 of itself, so are scores' parts
    and values; errors of signs that differ leave a few hundredths of the output's norm.
    """
    g = torch.Generator(device="cuda").manual_seed(0)
    hidden, q_heads, kv_heads, dim, page = 512, 8, 2, 64, 16
    lens, new = [40, 23], [3, 1]
    total = sum(lens) + sum(new)
    x = torch.randn(total, hidden, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn((q_heads + 2 * kv_heads) * dim, hidden, generator=g, device="cuda").mul(hidden ** -0.5).to(torch.bfloat16)
    scale = 1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")
    turns = moe.moe_rope_turns(dim, base=1e4, device="cuda")
    cache = moe.KvCache(12, kv_heads, page, dim)
    table, free = torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), torch.arange(12, dtype=torch.int32, device="cuda")
    context, head = ints([0, 0]), ints([0])
    outs = []
    for query, rows in ((lens, x[:sum(lens)]), (new, x[sum(lens):])):
        n = sum(query)
        start, seq, counts = ints([0] * 3), ints([0, 0]), ints([0] * 4)
        positions, slots = ints([0] * n), torch.zeros(n, dtype=torch.int64, device="cuda")
        moe.moe_kv_plan(context, ints(query), page, table, free, head, start, seq, positions, slots, counts)
        h = torch.empty_like(rows)
        moe.moe_norm(rows, scale, h)
        qkv = (h @ w.t()).view(n, -1, dim)
        q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + kv_heads], qkv[:, q_heads + kv_heads:]
        moe.moe_rope(positions, turns, q, k)
        cache.append(k, v, slots)
        outs.append(cache.attend(q, table, start, seq))
        context, head = seq, counts[1:2]
    assert cache.status() == moe.MOE_OK
    # The formula.
    f = x.double()
    f = f / torch.sqrt(f.square().mean(-1, keepdim=True) + 1e-6) * scale.double()
    qkv = (f @ w.double().t()).view(total, -1, dim)
    order = list(range(40)) + list(range(63, 66)), list(range(40, 63)) + [66]
    for r, rows in enumerate(order):
        part = qkv[rows]
        pos = torch.arange(len(rows), device="cuda", dtype=torch.float64)
        angle = pos[:, None] * torch.tensor([1e4 ** (-2.0 * i / dim) for i in range(dim // 2)], dtype=torch.float64, device="cuda")
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        a, b = part[..., : dim // 2], part[..., dim // 2:]
        rot = torch.cat((a * c - b * s, b * c + a * s), -1)
        q, k, v = rot[:, :q_heads], rot[:, q_heads:q_heads + kv_heads], part[:, q_heads + kv_heads:]
        k, v = (t.repeat_interleave(q_heads // kv_heads, 1) for t in (k, v))
        scores = torch.einsum("qhd,khd->hqk", q, k) / math.sqrt(dim)
        scores = scores.masked_fill(pos[None, None, :] > pos[None, :, None], -math.inf)
        want = torch.einsum("hqk,khd->qhd", torch.softmax(scores, -1), v)
        got = torch.cat((outs[0][:40] if r == 0 else outs[0][40:], outs[1][:3] if r == 0 else outs[1][3:])).double()
        assert torch.linalg.norm(got - want) <= 0.06 * torch.linalg.norm(want)


@pytest.mark.gpu
def test_a_step_from_norm_to_experts_in_a_graph(moe):
    """Norm, rope, append, shared attention, norm into the layer's plan, routing and experts, captured once and replayed."""
    import workload

    g = torch.Generator(device="cuda").manual_seed(1)
    tokens, hidden, q_heads, kv_heads, dim, page = 6, 256, 8, 2, 64, 16
    layer = moe.MoeLayer(tuple(torch.from_numpy(w).cuda() for w in workload.make_weights(32, hidden, 64, seed13=1, seed2=2)))
    cache = moe.KvCache(64, kv_heads, page, dim)
    for t in cache.tensors[:2]:
        t.copy_((torch.randn(t.shape, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn).view(torch.uint8))
    for t in cache.tensors[2:]:
        t.fill_(120)
    table = torch.arange(tokens, device="cuda").mul(5)[:, None].add(torch.arange(8, device="cuda")).int()
    table[:, :3] = ints([40, 41, 42])  # 48 shared tokens
    table = table.contiguous()
    lens, ones, free, head = torch.full((tokens,), 60, dtype=torch.int32, device="cuda"), ints([1] * tokens), ints([50]), ints([0])
    x = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    wq = torch.randn((q_heads + 2 * kv_heads) * dim, hidden, generator=g, device="cuda").mul(hidden ** -0.5).to(torch.bfloat16)
    wo = torch.randn(hidden, q_heads * dim, generator=g, device="cuda").mul(0.05).to(torch.bfloat16)
    gate = torch.randn(32, hidden, generator=g, device="cuda").mul(hidden ** -0.5).to(torch.bfloat16)
    turns, scale = moe.moe_rope_turns(dim, device="cuda"), torch.ones(hidden, device="cuda")
    scratch = torch.empty(moe.moe_kv_shared_bytes(tokens, q_heads, dim), dtype=torch.uint8, device="cuda")
    group_start, prefix = ints([0, tokens]), ints([48])

    def step(shared):
        start, seq, counts = torch.empty(tokens + 1, dtype=torch.int32, device="cuda"), torch.empty_like(lens), torch.empty(4, dtype=torch.int32, device="cuda")
        positions, slots = torch.empty_like(lens), torch.empty(tokens, dtype=torch.int64, device="cuda")
        moe.moe_kv_plan(lens, ones, page, table, free, head, start, seq, positions, slots, counts)
        h, residual = torch.empty_like(x), torch.empty_like(x)
        moe.moe_norm(x, scale, h)
        qkv = (h @ wq.t()).view(tokens, -1, dim)
        q, k, v = qkv.split([q_heads, kv_heads, kv_heads], dim=1)
        moe.moe_rope(positions, turns, q, k)
        cache.append(k, v, slots)
        if shared:
            attended = cache.attend_shared(q, table, start, seq, group_start, prefix, scratch=scratch, least_tiles=1)
        else:
            attended = cache.attend(q, table, start, seq)
        moe.moe_norm_quantize(layer.handle, attended.view(tokens, -1) @ wo.t(), scale, h, residual=x, residual_out=residual)
        ids, weights = torch.empty(tokens, 16, dtype=torch.int32, device="cuda"), torch.empty(tokens, 16, device="cuda")
        moe.moe_route(h @ gate.t(), ids, weights)
        rows = torch.empty(tokens, 16, hidden, dtype=torch.bfloat16, device="cuda")
        moe.moe_group(layer.handle, ids, tokens)
        moe.moe_experts(layer.handle, rows, tokens)
        return residual + (rows.float() * weights[..., None]).sum(1).to(torch.bfloat16), counts

    step(True)  # warm: loads kernels and libraries
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, counts = step(True)
    for seed in (3, 4):
        x.copy_(torch.randn(tokens, hidden, generator=g, device="cuda"))
        graph.replay()
        got = y.clone()
        again, _ = step(True)
        assert torch.equal(got, again)
        apart, _ = step(False)
        # The two attentions differ by roundings to BF16, which may move a code of the plan by one place in sixteen.
        assert torch.linalg.norm(got.float() - apart.float()) <= 0.02 * torch.linalg.norm(apart.float())
        assert counts[3].item() == 0
    assert cache.status() == moe.MOE_OK and moe.moe_sync_status(layer.handle) == moe.MOE_OK
    layer.close()


@pytest.mark.gpu
def test_example_with_samples_runs_and_equals_requests_of_their_own(moe):
    ex = example()
    y = ex.main(["--steps", "3", "--requests", "3", "--prompt", "45", "--samples", "4"])
    assert y.shape == (12, 256) and torch.isfinite(y.float()).all()
    # Two samples of one prompt, and the same as requests that read the prompt each.
    layer = ex.DecoderLayer(32, 256, 64, 8, 2, 64, pages=32, page_tokens=16)
    gen = torch.Generator().manual_seed(5)
    prompt, nexts = (torch.randn(n, 256, generator=gen).to(torch.bfloat16).cuda() for n in (37, 2))
    ones = ints([1, 1])
    forked = ex.Requests(1, 4, 32, 16)
    layer(prompt, forked.plan(ints([37]), 37))
    forked.fork(2, [layer.cache])
    got = layer(nexts, forked.plan(ones, 2))
    assert forked.block_table[0, 0] == forked.block_table[1, 0] and forked.block_table[0, 2] != forked.block_table[1, 2]
    own = ex.Requests(2, 4, 32, 16)
    layer(torch.cat((prompt, prompt)), own.plan(ints([37, 37]), 74))
    want = layer(nexts, own.plan(ones, 2))
    assert (got.float() - want.float()).norm() <= 0.05 * want.float().norm()
    layer.experts.close()
