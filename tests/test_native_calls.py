"""The Python calls that go from tensors to the C entries natively (csrc/tensors.cpp): taken, and as the package's own checks take them.

A call on the current stream goes natively where its tensors are what the entry
needs; with a stream given it goes by the package's checks. Both give the same bits.
"""
from __future__ import annotations

import pytest
import torch
from test_shared import Batch, moe, same  # noqa: F401


@pytest.fixture()
def native(moe, monkeypatch):  # noqa: F811
    """The statuses that the native functions answer, None where they decline."""
    inner, answers = moe._native or moe._use_torch(), []

    class Recorder:
        def __getattr__(self, name):
            def call(*args):
                answers.append(getattr(inner, name)(*args))
                return answers[-1]
            return call

    monkeypatch.setattr(moe, "_native", Recorder())
    return answers


def tuple_batch(moe, groups, *args, **kwargs):  # noqa: F811
    b = Batch(moe, groups, *args, **kwargs)
    b.cache = tuple(b.cache)
    return b


@pytest.mark.gpu
@pytest.mark.parametrize("rows,q_heads,dim", [(1, 16, 64), (4, 14, 128), (60, 4, 128), (3, 4, 256)])
@pytest.mark.parametrize("scale", [None, 0.05])
def test_shared_goes_natively_and_gives_the_same_bits(moe, native, rows, q_heads, dim, scale):  # noqa: F811
    b = tuple_batch(moe, [(640, same(5, rows + 30, rows)), (200, same(2, rows + 70, rows))], 16, 2, dim, q_heads, seed=dim + rows)
    got = b.check(b.run(scale=scale), scale)
    assert native == [moe.MOE_OK]
    stream = torch.cuda.current_stream()
    want = b.run(scale=scale, stream=stream)
    assert len(native) == 1 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # Rows of a fused projection, and no log-sum-exp.
    fused = torch.randn(b.q.shape[0], q_heads + 5, dim, device="cuda").to(torch.bfloat16)
    fused[:, 3:3 + q_heads] = b.q
    out = torch.full_like(b.q, 7.0)
    scratch = torch.empty(moe.moe_kv_shared_bytes(*b.q.shape), dtype=torch.uint8, device="cuda")
    moe.moe_kv_attend_shared(b.cache, fused[:, 3:3 + q_heads], b.table, b.start, b.lens, b.group_start, b.prefix_lens, out, b.workspace,
                             scratch, scale=scale, least_tiles=1)
    assert native == [moe.MOE_OK] * 2 and torch.equal(out, got[0])
    # Lists, and a table that is a part of a wider one.
    b.cache, wide = list(b.cache), torch.full((len(b.seq), b.table.shape[1] + 9), -1, dtype=torch.int32, device="cuda")
    wide[:, 4:4 + b.table.shape[1]] = b.table
    want = b.run(scale=scale)
    assert native[2] is None and torch.equal(got[0], want[0])
    b.cache, b.table = tuple(b.cache), wide[:, 4:4 + b.table.shape[1]]
    want = b.run(scale=scale)
    assert native[3] == moe.MOE_OK and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_shared_native_refusals(moe, native):  # noqa: F811
    b = tuple_batch(moe, [(200, same(5, 30))], 64, 2, 128, 8, seed=12, pad=0)
    k, v, ks, vs = b.cache
    out = torch.empty(b.q.shape, dtype=torch.bfloat16, device="cuda")
    scratch = torch.empty(moe.moe_kv_shared_bytes(*b.q.shape), dtype=torch.uint8, device="cuda")
    lse = torch.empty(b.q.shape[:2], device="cuda")
    good = dict(cache=b.cache, q=b.q, block_table=b.table, query_start=b.start, seq_lens=b.lens, group_start=b.group_start,
                prefix_lens=b.prefix_lens, out=out, workspace=b.workspace, scratch=scratch, lse=lse)
    for name, bad in (("scratch", scratch[:-1]), ("scratch", scratch.cpu()), ("workspace", b.workspace[:-1]), ("group_start", b.group_start[:1]),
                      ("group_start", b.group_start.long()), ("prefix_lens", b.prefix_lens.cpu()), ("out", out.float()), ("q", b.q.float()),
                      ("q", b.q[..., :64]), ("q", b.q[..., 1:]), ("query_start", b.start[1:]), ("block_table", b.table.long()),
                      ("block_table", b.table[:-1]), ("block_table", b.table.t()), ("seq_lens", b.lens[:-1]), ("out", out[:-1]), ("lse", lse[:, :-1]),
                      ("lse", lse.double()), ("cache", (k, v, ks)), ("cache", (k, v[:-1], ks, vs)), ("cache", (k, v, ks, vs.int())),
                      ("cache", (k.cpu(), v, ks, vs)), ("least_tiles", -1), ("scale", float("nan"))):
        with pytest.raises((moe.MoeError, ValueError, TypeError)) as e:
            moe.moe_kv_attend_shared(**dict(good, **{name: bad}))
        assert not isinstance(e.value, moe.MoeError) or e.value.code == moe.MOE_ERR_ARG
    # What the entry refuses is refused natively too: with tensors that fit, none declined.
    native.clear()
    with pytest.raises(moe.MoeError):
        moe.moe_kv_attend_shared(**dict(good, scale=float("inf")))
    assert native == [moe.MOE_ERR_ARG]
    moe.moe_kv_attend_shared(**good)
    assert native[1:] == [moe.MOE_OK]


@pytest.mark.gpu
def test_the_smaller_operators_go_natively_and_give_the_same_bits(moe, native):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(1)
    stream = torch.cuda.current_stream()

    def ints(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def both(call, *outputs):
        """The outputs of the native call, then of the other, which have to be the same."""
        for t in outputs:
            t.fill_(3)
        call(None)
        assert native.pop() == moe.MOE_OK and not native
        first = [t.clone() for t in outputs]
        for t in outputs:
            t.fill_(3)
        call(stream)
        assert not native
        for a, t in zip(first, outputs):
            assert torch.equal(a, t)

    x = torch.randn(9, 96, generator=g, device="cuda").to(torch.bfloat16)
    residual, w = torch.randn(9, 128, generator=g, device="cuda")[:, :96], torch.randn(96, generator=g, device="cuda")
    out, to = torch.empty_like(x), torch.empty(9, 96, device="cuda")
    codes, scales = torch.empty(9, 96, dtype=torch.uint8, device="cuda"), torch.empty(9, 3, dtype=torch.uint8, device="cuda")
    both(lambda s: moe.moe_norm(x, w, out, 1e-5, residual, to, codes, scales, 1.0, stream=s), out, to, codes, scales)
    both(lambda s: moe.moe_norm(x, w, out, stream=s), out)
    both(lambda s: moe.moe_norm(x, w, residual_out=to, codes=codes, scales=scales, stream=s), to, codes, scales)

    turns, positions = moe.moe_rope_turns(32, device="cuda"), ints(5, 0, 2 ** 31 - 1)
    qkv = torch.randn(3, 7, 64, generator=g, device="cuda").to(torch.bfloat16)
    q_out, k_out = torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    both(lambda s: moe.moe_rope(positions, turns, qkv[:, :4], qkv[:, 4:6], q_out, k_out, True, 1.5, stream=s), q_out, k_out)
    both(lambda s: moe.moe_rope(positions, turns, qkv[:, :4], q_out=q_out, stream=s), q_out)

    table, free, lens = ints(*range(12)).view(2, 6), torch.arange(12, 40, dtype=torch.int32, device="cuda"), ints(90, 33)
    out_table, out_lens, moves, counts = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((4, 6), (4,), (4, 3), (4,)))
    both(lambda s: moe.moe_kv_fork(ints(0, 1, 0, -1), table, lens, 16, free, ints(2), out_table, out_lens, moves, counts, stream=s),
         out_table, out_lens, moves, counts)
    pool, room = torch.empty(40, dtype=torch.int32, device="cuda"), torch.empty(moe.moe_kv_reclaim_bytes(40), dtype=torch.uint8, device="cuda")
    both(lambda s: moe.moe_kv_reclaim(table, lens, 16, pool, counts, room, stream=s), pool, counts)
    packed, leaving = torch.empty_like(table), torch.empty(20, 3, dtype=torch.int32, device="cuda")
    both(lambda s: moe.moe_kv_reclaim(table + 25, lens, 16, pool, counts, room, packed, leaving, stream=s), pool, counts, packed, leaving)

    cache = tuple(torch.randint(0, 256, s, generator=g, dtype=torch.uint8, device="cuda") for s in ((6, 2, 16, 64), (6, 2, 16, 64), (6, 2), (6, 2)))
    some = torch.tensor([[0, 3, 16], [1, 4, 5], [2, 5, 16]], dtype=torch.int32, device="cuda")
    for count in (None, ints(2)):
        parts = [tuple(t.clone() for t in cache) for _ in range(2)]
        moe.moe_kv_copy(parts[0], some, count)
        assert native.pop() == moe.MOE_OK
        moe.moe_kv_copy(parts[1], some, count, stream=stream)
        assert not native and all(torch.equal(a, b) for a, b in zip(*parts)) and not torch.equal(parts[0][0], cache[0])


@pytest.mark.gpu
def test_shared_on_another_stream_gives_the_replayed_graphs_bits(moe):  # noqa: F811
    """The inputs and lengths of the last replay, on a stream of their own."""
    b = tuple_batch(moe, [(500, same(6, 60)), (300, same(3, 80))], 64, 2, 128, 16, seed=10, pad=0)
    full = b.lens.clone()
    out, lse = torch.zeros_like(b.q), torch.zeros(b.q.shape[:2], device="cuda")
    scratch = torch.zeros(moe.moe_kv_shared_bytes(*b.q.shape), dtype=torch.uint8, device="cuda")
    args = (b.cache, b.q, b.table, b.start, b.lens, b.group_start, b.prefix_lens, out, b.workspace, scratch, lse, None, 1)
    moe.moe_kv_attend_shared(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_kv_attend_shared(*args)
    side = torch.cuda.Stream()
    for step in range(3):
        b.lens.copy_(full - 7 * step)
        b.prefix_lens.copy_(torch.tensor([500 - 64 * step, 300 if step != 1 else 0]))
        graph.replay()
        other, other_lse, room = torch.full_like(out, 7.0), torch.full_like(lse, 7.0), torch.empty_like(scratch)
        side.wait_stream(torch.cuda.current_stream())  # (its inputs, and the workspace)
        moe.moe_kv_attend_shared(*args[:7], other, b.workspace, room, other_lse, None, 1, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(other, out) and torch.equal(other_lse, lse)
        b.check((other, other_lse))


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hidden", [(1, 3584), (700, 3584), (5, 1000), (3, 640)])
def test_norm_repeats_itself(moe, tokens, hidden):  # noqa: F811
    x, r = (torch.randn(tokens, hidden, device="cuda").to(torch.bfloat16) for _ in range(2))
    w, first = torch.randn(hidden, device="cuda"), None
    for _ in range(20):
        out, to = torch.empty_like(x), torch.empty_like(x)
        moe.moe_norm(x, w, out, residual=r, residual_out=to)
        first = first or (out, to)
        assert torch.equal(out, first[0]) and torch.equal(to, first[1])
