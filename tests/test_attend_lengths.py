"""moe_kv_attend and moe_kv_attend_shared at the ends of the lengths' range.

A query of a length of 0 or below stands before its sequence and sees nothing, so
such a length gives the bits that 0 gives. The longest sequences hold keys of
zero and nearly everywhere values of 2: every weight is 1 and every sum of a CTA
an even number below 2^25, which FP32 holds, so only the join of the CTAs' sums
and the division round (under 2^-20 in all), and the output once, under 2^-8.
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


def long_cache(page, dim):
    """Three pages of zero keys: values of 2 in page 0, of -3 in page 1, of 5 in page 2."""
    k = torch.zeros(3, 1, page, dim, dtype=torch.uint8, device="cuda")
    v = torch.empty_like(k)
    for p, value in enumerate((2.0, -3.0, 5.0)):
        v[p] = torch.tensor(value).to(torch.float8_e4m3fn).view(torch.uint8).item()
    ones = torch.full((3, 1), 127, dtype=torch.uint8, device="cuda")
    return [k, v, ones, ones.clone()]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim", [(1, 64), (100, 128)])
def test_the_longest_sequence(moe, rows, dim):  # noqa: F811
    """2^31 - 1 tokens, whose last tile ends where the lengths do: page 0 but for its first entry (page 1) and last (page 2)."""
    page, most = 128, 2 ** 31 - 1
    cache = long_cache(page, dim)
    table = torch.zeros(1, 2 ** 31 // page, dtype=torch.int32, device="cuda")
    table[0, 0], table[0, -1] = 1, 2
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn(rows, 1, dim, device="cuda").to(torch.bfloat16)
    out, lse = torch.full_like(q, 7.0), torch.full((rows, 1), 7.0, device="cuda")
    workspace = torch.zeros(moe.MOE_KV_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    for window, value in ((0, 2.0), (50, 5.0)):
        moe.moe_kv_attend(cache, q, table, ints(0, rows), ints(most), out, workspace, lse=lse, window=window)
        assert moe.moe_kv_sync_status(workspace) == moe.MOE_OK
        # Rows of the window's first tile see its tokens and those of the last page.
        seen = torch.arange(most - rows, most, device="cuda").double() + 1 if not window else torch.full((rows,), 50.0, device="cuda").double()
        want = torch.full((rows,), value, device="cuda").double()
        if window:  # tokens of the last page: from 2^31 - 128 on
            in_last = (torch.arange(most - rows, most, device="cuda") - (2 ** 31 - 128) + 1).clamp(0, 50).double()
            want = (5.0 * in_last + 2.0 * (50 - in_last)) / 50
        assert ((lse[:, 0].double() - seen.log()).abs() <= 1e-5).all()
        assert ((out[:, 0].double() - want[:, None]).abs() <= 2.0 ** -8 * want[:, None].abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim", [(1, 64), (60, 128)])
def test_the_longest_shared_prefix(moe, rows, dim):  # noqa: F811
    """Two requests of 2^31 - 1 tokens that share all pages but the last: the prefix's last tile ends inside 2^31."""
    page, most = 64, 2 ** 31 - 1
    cache = tuple(long_cache(page, dim))
    table = torch.zeros(2, 2 ** 31 // page, dtype=torch.int32, device="cuda")
    table[:, 0], table[0, -1], table[1, -1] = 1, 2, 1
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn(2 * rows, 1, dim, device="cuda").to(torch.bfloat16)
    out, lse = torch.full_like(q, 7.0), torch.full((2 * rows, 1), 7.0, device="cuda")
    workspace = torch.zeros(moe.MOE_KV_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    scratch = torch.empty(moe.moe_kv_shared_bytes(*q.shape), dtype=torch.uint8, device="cuda")
    moe.moe_kv_attend_shared(cache, q, table, ints(0, rows, 2 * rows), ints(most, most), ints(0, 2), ints(most), out, workspace, scratch,
                             lse=lse, least_tiles=1)
    assert moe.moe_kv_sync_status(workspace) == moe.MOE_OK
    seen = (torch.arange(most - rows, most, device="cuda").double() + 1).repeat(2)
    assert ((lse[:, 0].double() - seen.log()).abs() <= 1e-5).all()
    assert ((out.double() - 2.0).abs() <= 2.0 ** -7).all()
