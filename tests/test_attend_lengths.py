"""moe_kv_attend and moe_kv_attend_shared at the ends of the lengths' range.

A query of a length of 0 or below stands before its sequence and sees nothing, so
such a length gives the bits that 0 gives.
"""
from __future__ import annotations

import pytest
import torch
from test_shared import Batch, moe, same  # noqa: F401

SHAPES = [(1, 8, 64), (1, 8, 128), (3, 14, 256), (20, 14, 64), (50, 4, 64), (50, 4, 128), (300, 2, 128)]  # query rows, heads, dim


def attend(moe, b, window=0):  # noqa: F811
    out, lse = torch.full_like(b.q, 7.0), torch.full(b.q.shape[:2], 7.0, device="cuda")
    moe.moe_kv_attend(b.cache, b.q, b.table, b.start, b.lens, out, b.workspace, lse=lse, window=window)
    return out, lse


@pytest.mark.gpu
@pytest.mark.parametrize("rows,q_heads,dim", SHAPES)
@pytest.mark.parametrize("length", [-1, -5, -2 ** 31 + 1, -2 ** 31])
def test_lengths_below_zero_see_nothing(moe, length, rows, q_heads, dim):  # noqa: F811
    b = Batch(moe, [(640, same(4, rows + 20, rows)), (320, same(3, rows + 150, rows))], 16, 2, dim, q_heads, seed=rows)
    first, last = b.start[1].item(), b.start[2].item()
    calls = [b.run, lambda: b.run(least=0), lambda: attend(moe, b), lambda: attend(moe, b, 100)]
    b.lens[1] = 0
    want = [f() for f in calls]
    b.lens[1] = length
    for f, (out, lse) in zip(calls, want):
        got, got_lse = f()
        assert not got[first:last].any() and torch.isneginf(got_lse[first:last]).all()
        assert torch.equal(got, out) and torch.equal(got_lse, lse)
    b.check()
