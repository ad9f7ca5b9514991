"""moe_kv_attend_shared against attention in 64 bits, request by request.

Tolerances, derived before their first run: weights are held within 2^-16 of
themselves, queries within 2^-21 of their row's largest element (a score within
1e-5 at these sizes), sums are FP32 and the two parts are joined in FP32: less
than 2^-12 of sum_j w_j |v_j| in all; the output is rounded to BF16 once, half a
step or 2^-8 of it. The log-sum-exp is FP32 with scores of |s| <= 40: 1.6e-4
bounds it; 2e-5 is asked of scores under 12.
"""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__

    __graft_entry__.build()
    import mxfp4_weight_mxfp8_gb300 as moe

    return moe


# ------------------------------------------------------------------- refusals
def call(moe, cache=None, batch=None, prefixes=None, **changes):
    c = moe._KvCache(k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x40000, pages=4, page_tokens=16, kv_heads=2, head_dim=64)
    b = moe._KvBatch(block_table=0x50000, table_stride=8, query_start=0x60000, seq_lens=0x70000, table_width=8, requests=4, tokens=4)
    p = moe._KvPrefixes(group_start=0x80000, prefix_lens=0x90000, groups=2)
    for block, more in ((c, cache), (b, batch), (p, prefixes)):
        for k, v in (more or {}).items():
            setattr(block, k, v)
    args = dict(q=0xA0000, token=256, head=64, q_heads=4, scale=0.1, out=0xB0000, lse=None, workspace=0xC0000, scratch=0xD0000)
    args.update(changes)
    p_ref = None if args.pop("no_prefixes", False) else ctypes.byref(p)
    return moe.library().moe_kv_attend_shared(ctypes.byref(c), ctypes.byref(b), p_ref, args["q"], args["token"], args["head"], args["q_heads"],
                                              args["scale"], args["out"], args["lse"], args["workspace"], args["scratch"], None)


@pytest.mark.parametrize("changes", [
    dict(cache=dict(k=0)), dict(cache=dict(head_dim=96)), dict(batch=dict(requests=0)), dict(batch=dict(requests=1025)), dict(batch=dict(tokens=-1)),
    dict(batch=dict(table_stride=7)), dict(batch=dict(block_table=0)), dict(batch=dict(query_start=0x60002)), dict(q_heads=3), dict(q_heads=0),
    dict(token=4), dict(head=-8), dict(scale=math.inf), dict(q=0), dict(q=0xA0008), dict(out=0), dict(workspace=0), dict(workspace=0xC0008),
    dict(lse=0xE0002), dict(no_prefixes=True), dict(prefixes=dict(groups=0)), dict(prefixes=dict(groups=5)), dict(prefixes=dict(group_start=0)),
    dict(prefixes=dict(prefix_lens=0)), dict(prefixes=dict(least_tiles=-1)), dict(prefixes=dict(prefix_lens=0x90001)), dict(scratch=0), dict(scratch=0xD0004)])
def test_shared_refusals(moe, changes):
    assert call(moe, **changes) == moe.MOE_ERR_ARG
    assert moe.moe_last_error_detail()


def test_shared_of_no_tokens_is_no_work(moe):
    assert call(moe, batch=dict(tokens=0), scratch=None, q=0) == moe.MOE_OK


def test_shared_bytes(moe):
    assert moe.moe_kv_shared_bytes(0, 1, 64) == moe.MOE_KV_SHARED_HEADER
    assert moe.moe_kv_shared_bytes(3, 8, 128) == moe.MOE_KV_SHARED_HEADER + 3 * 8 * 129 * 4
    assert moe.moe_kv_shared_bytes(100000, 1024, 256) == moe.MOE_KV_SHARED_HEADER + 100000 * 1024 * 257 * 4
    for bad in ((-1, 1, 64), (1, 0, 64), (1, 1025, 64), (1, 1, 80)):
        assert moe.moe_kv_shared_bytes(*bad) == 0


# ------------------------------------------------------------------- numerics
class Batch:
    """Groups [(prefix, [(tokens behind it, query rows), ...]), ...] on the GPU; unused rows and pages hold NaN."""

    def __init__(self, moe, groups, page, heads, dim, q_heads, seed=0, pad=2, spread=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.moe, self.page, self.dim = moe, page, dim
        rows = [(p + s if s or n else 0, n, i) for i, (p, requests) in enumerate(groups) for s, n in requests]
        self.seq = [t for t, _, _ in rows]
        self.new = [n for _, n, _ in rows]
        self.prefix = [p for p, _ in groups]
        starts = np.cumsum([0] + [len(r) for _, r in groups])
        width = max(max(-(-t // page) for t in self.seq), 1) + 2
        pages = sum(-(-t // page) for t in self.seq) + sum(p // page for p in self.prefix) + 3
        ids, at, table = rng.permutation(pages), 0, np.full((len(rows), width), -1, np.int32)
        k = torch.full((pages, heads, page, dim), 0x7F, dtype=torch.uint8, device="cuda")
        v = torch.full_like(k, 0x7F)
        for i, (p, requests) in enumerate(groups):
            common = ids[at:at + p // page]
            at += p // page
            for r in range(starts[i], starts[i + 1]):
                n = -(-self.seq[r] // page)
                c = min(len(common), n)
                table[r, :c] = common[:c]
                table[r, c:n] = ids[at:at + n - c]
                at += n - c
                if not self.seq[r]:
                    table[r] = rng.integers(0, pages, width)  # a row that holds nothing may name anything
        for r, t in enumerate(self.seq):
            for j in range(-(-t // page)):
                n = min(page, t - j * page)
                for c in (k, v):
                    c[table[r, j], :, :n] = (torch.randn(heads, n, dim, generator=g, device="cuda") * 60 * spread).clamp(-448, 448) \
                        .to(torch.float8_e4m3fn).view(torch.uint8)
        scales = [torch.randint(117, 124, (pages, heads), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
        self.cache = [k, v, *scales]
        self.table = torch.from_numpy(table).cuda()
        self.start = torch.tensor(np.cumsum([0] + self.new), dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(self.seq, dtype=torch.int32, device="cuda")
        self.group_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.prefix_lens = torch.tensor(self.prefix, dtype=torch.int32, device="cuda")
        self.q = (torch.randn(sum(self.new) + pad, q_heads, dim, generator=g, device="cuda") * 1.3).to(torch.bfloat16)
        self.workspace = torch.zeros(moe.MOE_KV_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")

    def run(self, scratch=None, scale=None, stream=None, least=1):  # least 1: shared whatever that saves
        out = torch.full(self.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        if scratch is None:  # NaN where nothing has been written
            scratch = torch.full((self.moe.moe_kv_shared_bytes(*self.q.shape),), 0xFF, dtype=torch.uint8, device="cuda")
        self.moe.moe_kv_attend_shared(self.cache, self.q, self.table, self.start, self.lens, self.group_start, self.prefix_lens, out,
                                      self.workspace, scratch, lse=lse, scale=scale, least_tiles=least, stream=stream)
        return out, lse

    def reference(self, scale=None):
        k, v, ks, vs = self.cache
        heads, q_heads = k.shape[1], self.q.shape[1]
        out = torch.zeros(self.q.shape, dtype=torch.float64, device="cuda")
        lse = torch.full(self.q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        mass = torch.zeros_like(out)
        start, lens, pages = self.start.tolist(), self.lens.tolist(), k.shape[0]
        for r in range(len(lens)):
            a, b, n = start[r], start[r + 1], min(max(lens[r], 0), self.table.shape[1] * self.page)
            if a == b:
                continue
            entries = self.table[r, : -(-n // self.page)].long()
            there = ((entries >= 0) & (entries < pages)).repeat_interleave(self.page)[:n]
            entries = entries.clamp(0, pages - 1)

            def rows(c, s):
                x = c[entries].view(torch.float8_e4m3fn).double() * torch.exp2(s[entries].double() - 127)[:, :, None, None]
                return x.transpose(1, 2).reshape(-1, heads, self.dim)[:n].repeat_interleave(q_heads // heads, 1)

            keys, values = rows(k, ks), rows(v, vs)
            pos = lens[r] - (b - a) + torch.arange(b - a, device="cuda")
            seen = (torch.arange(n, device="cuda") <= pos[:, None]) & there
            used = seen.any(0)
            keys = torch.where(used[:, None, None], keys, 0.0)
            values = torch.where(used[:, None, None], values, 0.0)
            s = torch.einsum("qhd,khd->qhk", self.q[a:b].double(), keys) * (scale or self.dim ** -0.5)
            s = s.masked_fill(~seen[:, None], -math.inf)
            lse[a:b] = torch.logsumexp(s, -1)
            w = torch.where(seen[:, None], torch.exp(s - lse[a:b, :, None].clamp(min=-1e30)), 0.0)
            out[a:b] = torch.einsum("qhk,khd->qhd", w, values)
            mass[a:b] = torch.einsum("qhk,khd->qhd", w, values.abs())
        return out, lse, mass

    def check(self, got=None, scale=None):
        out, lse = got or self.run(scale=scale)
        assert self.moe.moe_kv_sync_status(self.workspace) == self.moe.MOE_OK
        n = int(self.start[-1])
        assert (out[n:] == 7).all() and (lse[n:] == 7).all()
        want, want_lse, mass = self.reference(scale)
        out, lse, want, want_lse, mass = out[:n].double(), lse[:n].double(), want[:n], want_lse[:n], mass[:n]
        # A NaN that a row sees is in its results, and nowhere else.
        assert torch.equal(out.isnan(), want.isnan()) and torch.equal(lse.isnan(), want_lse.isnan())
        out, lse, want, want_lse, mass = (torch.where(x.isnan(), 0.0, x) for x in (out, lse, want, want_lse, mass))
        seen = want_lse > -math.inf
        assert torch.equal(lse[~seen], want_lse[~seen]) and not out[~seen].any()
        err = (lse[seen] - want_lse[seen]).abs()
        assert (err <= torch.where(want_lse[seen].abs() < 12, 2e-5, 1.6e-4)).all(), err.max()
        worst = (out - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -12 * mass + 1e-30)
        assert (worst <= 0).all(), worst.max()
        return got


def same(n, total, rows=1):
    return [(total, rows)] * n


CASES = [
    # page, dim, kv heads, query heads, groups
    (64, 128, 1, 1, [(64, same(2, 1))]),
    (64, 128, 8, 64, [(777, same(4, 40))]),                      # 32 rows to a group and head: the widest row tile
    (16, 64, 2, 2, [(50, same(3, 5)), (16, same(2, 1)), (15, same(2, 3)), (17, [(1, 1), (0, 0), (9, 2)])]),
    (16, 64, 1, 8, [(300, same(1, 20)), (400, same(5, 7)), (0, same(4, 33))]),
    (32, 256, 2, 14, [(500, same(3, 17)), (250, [(3, 3), (65, 65)])]),
    (128, 128, 4, 28, [(1300, [(1, 1), (129, 1), (0, 0), (5, 5)]), (127, same(3, 300)), (128, same(2, 1)), (255, same(2, 2))]),
    (64, 128, 2, 32, [(640, same(20, 70))]),                     # many rows over the prefix, few behind it
    (64, 64, 3, 9, [(1000, same(40, 3)), (200, same(7, 130, 3))]),
    (128, 256, 1, 16, [(600, same(20, 40)), (90, same(3, 100, 2))]),
    (64, 64, 1, 40, [(2000, same(3, 50, 9))]),
    (64, 128, 2, 16, [(1000, same(3, 300, 150)), (5, same(2, 90, 90))]),  # many rows in both
    (16, 64, 4, 28, [(700, same(2, 200, 200)), (333, [(150, 129), (1, 1)])]),
    (64, 128, 2, 8, [(20000, same(6, 10))]),                     # a prefix cut between many CTAs
    (64, 64, 1, 16, [(30000, same(30, 10))]),
    (32, 128, 1, 3, [(40, same(1, 10))] * 60),                   # nothing to share
    (16, 64, 1, 4, [(100, same(2, 2))] * 200),
    (64, 256, 1, 2, [(15000, same(8, 4000))]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("page,dim,heads,q_heads,groups", CASES)
def test_shared_matches_64_bits(moe, page, dim, heads, q_heads, groups):
    b = Batch(moe, groups, page, heads, dim, q_heads, seed=page + dim)
    first = b.run()
    b.check(first)
    # moe_kv_attend's but for the order of the sums; the same bits each time.
    out, lse = torch.full_like(first[0], 7), torch.full_like(first[1], 7)
    moe.moe_kv_attend(b.cache, b.q, b.table, b.start, b.lens, out, b.workspace, lse=lse)
    b.check((out, lse))
    for _ in range(3):
        again = b.run()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    # By the library's own rule, and nothing shared: moe_kv_attend's results, bit for bit.
    b.check(b.run(least=0))
    alone = b.run(least=2 ** 31 - 1)
    assert torch.equal(alone[0], out) and torch.equal(alone[1], lse)
    assert not b.workspace[:moe.MOE_KV_WORKSPACE_HEADER].any()


@pytest.mark.gpu
@pytest.mark.parametrize("prefix", [[-5, 0], [10 ** 6, 2 ** 31 - 1], [15, 16], [47, 48], [130, 129], [-2 ** 31, 1]])
def test_shared_prefix_lengths_are_held_to_what_all_see(moe, prefix):
    b = Batch(moe, [(160, [(3, 2), (0, 0), (40, 1), (1, 1)]), (144, same(3, 20, 3))], 16, 2, 64, 4, seed=3)
    b.prefix_lens.copy_(torch.tensor(prefix))
    # What both groups' tables share is what they shared at first; a longer claim is the caller's fault, so it stays within.
    b.prefix_lens.clamp_(max=144)
    b.check()


@pytest.mark.gpu
def test_shared_contexts_shorter_than_the_prefix(moe):
    """A request still inside the prefix (a chunk of it) holds the group's share to its own context."""
    b = Batch(moe, [(320, same(3, 30))], 16, 2, 64, 8, seed=4)
    b.lens[1] = 100  # in the middle of a page of the prefix, its query row among them
    b.check()
    b.lens[2] = 1
    b.check()
    b.lens[2] = 0  # a query row that stands before the sequence
    out, lse = b.check(b.run())
    assert not out[2].any() and torch.isneginf(lse[2]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("starts", [[0, 2, 4], [1, 2, 5], [0, 3, 2 ** 31 - 1], [0, -1, 5], [0, 5, 3], [5, 0, 5]])
def test_shared_groups_that_do_not_cover_the_requests_share_nothing(moe, starts):
    b = Batch(moe, [(100, same(2, 10)), (200, same(3, 20))], 16, 1, 64, 4, seed=5)
    b.group_start.copy_(torch.tensor(starts))
    got = b.check(b.run())
    out, lse = torch.full_like(got[0], 7), torch.full_like(got[1], 7)
    moe.moe_kv_attend(b.cache, b.q, b.table, b.start, b.lens, out, b.workspace, lse=lse)
    assert torch.equal(out, got[0]) and torch.equal(lse, got[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n,q_heads", [(1, 4), (4, 8), (50, 4)])
def test_shared_plan_that_shares_nothing_leaves_attends_bits(moe, dim, n, q_heads):
    """A table so wide that the call might save much, prefixes so short that it would not: decided on the device."""
    b = Batch(moe, [(200, [(5 + 61 * i % 90 + n, n) for i in range(12)]), (70, [(3 + n, n)] * 12)], 16, 2, dim, q_heads, seed=dim + n)
    b.table = torch.cat([b.table, torch.full((len(b.seq), 8000), -1, dtype=torch.int32, device="cuda")], 1)
    got = b.run(least=0)
    out, lse = torch.full_like(got[0], 7), torch.full_like(got[1], 7)
    moe.moe_kv_attend(b.cache, b.q, b.table, b.start, b.lens, out, b.workspace, lse=lse)
    assert torch.equal(out, got[0]) and torch.equal(lse, got[1])
    b.check(b.run())  # and shared, in spite of that


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [2, 40])
@pytest.mark.parametrize("change", [{0: -5}, {0: -2 ** 31}, {-1: 2 ** 31 - 1}, {0: -3, -1: 10 ** 6}, {-1: 0}, {-1: -7}, {-2: 10 ** 6}])
def test_shared_query_starts_out_of_range_are_what_they_are_to_attend(moe, change, rows):
    """Starts below 0 and past the tokens count as those; one that falls leaves its request no rows."""
    b = Batch(moe, [(160, [(9, rows)] * 2), (96, [(rows, rows), (70, rows), (80, rows)])], 16, 2, 64, 4, seed=21)
    for at, value in change.items():
        b.start[at] = value
    out, lse = b.run()
    want, want_lse = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    moe.moe_kv_attend(b.cache, b.q, b.table, b.start, b.lens, want, b.workspace, lse=want_lse)
    assert torch.equal((lse == 7.0), (want_lse == 7.0)) and torch.equal((out == 7.0).all(2), (want_lse == 7.0))
    # Each is half a step of BF16 and 2^-12 of sum_j w_j |v_j| <= 448 / 16 off, its log-sum-exp 1.6e-4.
    assert ((out.double() - want.double()).abs() <= 1.01 * (2.0 ** -7 * want.double().abs() + 2.0 ** -11 * 28)).all()
    assert ((lse - want_lse).abs()[want_lse != 7.0] <= 3.2e-4).all()


@pytest.mark.gpu
def test_shared_empty_groups_and_tables_with_holes(moe):
    b = Batch(moe, [(100, same(2, 10)), (200, same(3, 20))], 16, 1, 64, 4, seed=6)
    b.group_start = torch.tensor([0, 0, 2, 2, 5], dtype=torch.int32, device="cuda")
    b.prefix_lens = torch.tensor([50, 100, 70, 200], dtype=torch.int32, device="cuda")
    b.check()
    b.table[:2, 3] = -1        # a page of the prefix that is not there
    b.table[2:, 5] = 10 ** 6   # and one outside the cache
    b.table[3, 12] = -7
    b.check()
    b.lens[2:] = 10 ** 6       # longer than the table's rows
    b.check()


@pytest.mark.gpu
@pytest.mark.parametrize("q_heads,n", [(4, 2), (8, 4), (8, 20)])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("at", [0, 100, 330])
@pytest.mark.parametrize("byte", [121, 119])
def test_shared_dominant_token_without_value(moe, byte, at, dim, q_heads, n):
    """A token of large score and value zero, in the prefix or behind it: the others' weights are all of the output.

    Scores of about 80 nats at the larger scale put them under 2^-100 of the row's largest weight, where nothing is
    promised of them: up to 350 such weights of values up to 448 * 2^-4 are 2^-100 * 350 * 28 in the output. At the
    smaller scale they are about 20 nats under it.
    """
    b = Batch(moe, [(320, same(n, 30))], 64, 1, dim, q_heads, seed=7)
    for r in range(n if at >= 320 else 1):
        p = b.table[r, at // 64]
        b.cache[0][p, 0, at % 64] = 0x7E  # 448 in every element
        b.cache[2][p, 0] = byte
        b.cache[1][p, 0, at % 64] = 0
    b.q[:, :, :] = b.q.abs()
    out, lse = b.run()
    want, want_lse, mass = b.reference()
    m = n
    err = (out[:m].double() - want[:m]).abs()
    assert (err <= 2.0 ** -8 * want[:m].abs() + 2.0 ** -8 * mass[:m] + 2.0 ** -100 * 350 * 28).all()
    assert ((lse[:m].double() - want_lse[:m]).abs() <= 2.0 ** -20 * want_lse[:m].abs() + 2e-5).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 30])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_shared_nan_in_the_prefix_reaches_every_row_and_behind_it_its_own(moe, dim, n):
    b = Batch(moe, [(200, same(n, 30)), (200, same(2, 30))], 64, 1, dim, 4, seed=8)
    clean = b.run()[0]
    b.cache[1][b.table[0, 1], 0, 5, 9] = 0x7F     # the first group's prefix
    b.cache[1][b.table[n, 3], 0, 20, 11] = 0xFF   # behind the second group's, its first request's own page
    out = b.run()[0]
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[:n, :, 9] = True
    bad[n, :, 11] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])
    # A NaN in a query row is that row's alone, in both parts.
    b.q[1, 2, 3] = math.nan
    out, lse = b.run()
    assert torch.isnan(out[1, 2]).all() and torch.isnan(lse[1, 2])
    bad[1, 2] = True
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.gpu
def test_shared_prefix_after_forks(moe):
    """A prompt, samples forked from it, tokens of their own: plan, fork, copy, append and attention, against one request each."""
    page, heads, dim, q_heads, samples, prompt, steps = 16, 2, 64, 8, 5, 75, 20
    cache = moe.KvCache(64, heads, page, dim)
    g = torch.Generator(device="cuda").manual_seed(9)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def rows(n, h):
        return torch.randn(n, h, dim, generator=g, device="cuda").to(torch.bfloat16)

    def plan(lens, new, table, free, head, total):
        q_start, seq, counts = ints([0] * (len(new) + 1)), torch.empty_like(lens), ints([0] * 4)
        positions, slots = ints([0] * total), torch.zeros(total, dtype=torch.int64, device="cuda")
        moe.moe_kv_plan(lens, ints(new), page, table, free, head, q_start, seq, positions, slots, counts)
        return q_start, seq, slots, counts

    table, free = torch.full((1, 8), -1, dtype=torch.int32, device="cuda"), torch.arange(64, dtype=torch.int32, device="cuda")
    _, lens, slots, counts = plan(ints([0]), [prompt], table, free, ints([0]), prompt)
    cache.append(rows(prompt, heads), rows(prompt, heads), slots)
    out_table, out_lens, moves, forked = ints([[0] * 8] * samples), ints([0] * samples), ints([[0] * 3] * samples), ints([0] * 4)
    moe.moe_kv_fork(ints([0] * samples), table, lens, page, free, counts[1:2], out_table, out_lens, moves, forked)
    cache.copy(moves)
    assert forked.tolist() == [samples - 1, 5 + samples - 1, prompt, 0]
    table, lens, head = out_table, out_lens, forked[1:2]
    for _ in range(steps):
        q_start, lens, slots, counts = plan(lens, [1] * samples, table, free, head, samples)
        head = counts[1:2]
        cache.append(rows(samples, heads), rows(samples, heads), slots)
        q = rows(samples, q_heads)
        got, got_lse = cache.attend_shared(q, table, q_start, lens, ints([0, samples]), ints([prompt]), return_lse=True, least_tiles=1)
        want, want_lse = cache.attend(q, table, q_start, lens, return_lse=True)
        # Both are held to the tolerances of this file's head; between two of them twice that.
        assert (got.double() - want.double()).abs().max() <= 2 * (2.0 ** -8 * want.abs().max() + 2.0 ** -12 * 4)
        assert (got_lse - want_lse).abs().max() <= 4e-5
    assert cache.status() == moe.MOE_OK and counts[3].item() == 0
    # All samples' prompts are one's pages but the last; the others are their own.
    assert torch.equal(table[:, :4], table[:1, :4].expand(samples, 4)) and len(set(table[:, 4].tolist())) == samples


@pytest.mark.gpu
def test_shared_in_a_graph_with_new_lengths_and_on_a_stream(moe):
    b = Batch(moe, [(500, same(6, 60)), (300, same(3, 80))], 64, 2, 128, 16, seed=10, pad=0)
    full = b.lens.clone()
    out, lse = torch.zeros_like(b.q), torch.zeros(b.q.shape[:2], device="cuda")
    scratch = torch.zeros(moe.moe_kv_shared_bytes(*b.q.shape), dtype=torch.uint8, device="cuda")
    args = (b.cache, b.q, b.table, b.start, b.lens, b.group_start, b.prefix_lens, out, b.workspace, scratch, lse, None, 1)
    moe.moe_kv_attend_shared(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_kv_attend_shared(*args)
    for step in range(4):
        b.lens.copy_(full - 7 * step)
        b.prefix_lens.copy_(torch.tensor([500 - 64 * step, 0 if step == 2 else 300]))
        graph.replay()
        b.check((out.clone(), lse.clone()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = b.run(stream=side)
    side.synchronize()
    assert torch.equal(got[0], out) or step  # (the last step's lengths)
    b.check(got)
    c = moe.KvCache(1, 2, 64, 128)
    c.k, c.v, c.k_scale, c.v_scale = b.cache
    again, again_lse = c.attend_shared(b.q, b.table, b.start, b.lens, b.group_start, b.prefix_lens, return_lse=True, least_tiles=1, stream=side)
    side.synchronize()
    assert torch.equal(again, got[0]) and torch.equal(again_lse, got[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dim,n,other", [(64, 1, 40), (128, 1, 40), (64, 40, 2), (256, 2, 6), (128, 2, 1)])
def test_shared_two_calls_at_once(moe, dim, n, other):
    """On two streams, each with its own workspace and scratch: the bits of each alone."""
    batches = [Batch(moe, [(3000, [(20 + 70 * i % 300 + r, r) for i in range(14)]), (500, [(9 + r, r)] * 9)], 16, 2, dim, 8, seed=r)
               for r in (n, other)]
    alone = [b.run() for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    room = [[torch.empty(moe.moe_kv_shared_bytes(*b.q.shape), dtype=torch.uint8, device="cuda"), *(torch.empty_like(x) for x in a)]
            for b, a in zip(batches, alone)]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, s, (scratch, out, lse) in zip(batches, streams, room):
            with torch.cuda.stream(s):
                out.fill_(7.0), lse.fill_(7.0)
                moe.moe_kv_attend_shared(b.cache, b.q, b.table, b.start, b.lens, b.group_start, b.prefix_lens, out, b.workspace, scratch,
                                         lse=lse, least_tiles=1)
    torch.cuda.synchronize()
    for b, (want, want_lse), (_, out, lse) in zip(batches, alone, room):
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert not b.workspace[:moe.MOE_KV_WORKSPACE_HEADER].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dim,n,rows", [(64, 4, 1), (128, 4, 1), (256, 4, 1), (128, 40, 1), (64, 40, 1), (128, 3, 50)])
@pytest.mark.parametrize("cta", [1, 5])
def test_shared_waits_that_run_out(moe, dim, n, rows, cta):
    """A CTA's first tile never comes, in the prefix's launch and then in the requests': reported, and the next call right."""
    b = Batch(moe, [(3000, same(n, 500 + rows, rows))], 64, 2, dim, 16, seed=11)
    want = b.check(b.run())
    for _ in range(2):
        moe.moe_kv_set_timeout(b.workspace, 1_000_000)
        moe.moe_kv_debug_withhold(b.workspace, cta)
        b.run()
        assert moe.moe_kv_sync_status(b.workspace) == moe.MOE_ERR_DEVICE_TIMEOUT
        got = b.run()
        assert moe.moe_kv_sync_status(b.workspace) == moe.MOE_OK
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.gpu
def test_shared_strided_queries_and_python_refusals(moe):
    b = Batch(moe, [(200, same(5, 30))], 64, 2, 128, 8, seed=12, pad=0)
    want = b.check(b.run())
    fused = torch.zeros(b.q.shape[0], 20, 128, dtype=torch.bfloat16, device="cuda")
    fused[:, 3:11] = b.q
    b.q = fused[:, 3:11]
    got = b.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = torch.empty(b.q.shape, dtype=torch.bfloat16, device="cuda")
    scratch = torch.empty(moe.moe_kv_shared_bytes(*b.q.shape), dtype=torch.uint8, device="cuda")
    good = dict(cache=b.cache, q=b.q, block_table=b.table, query_start=b.start, seq_lens=b.lens, group_start=b.group_start,
                prefix_lens=b.prefix_lens, out=out, workspace=b.workspace, scratch=scratch)
    for name, bad in (("scratch", scratch[:-1]), ("scratch", scratch.cpu()), ("workspace", b.workspace[:-1]), ("group_start", b.group_start[:1]),
                      ("group_start", b.group_start.long()), ("prefix_lens", b.prefix_lens.cpu()), ("out", out.float()), ("q", b.q.float()),
                      ("query_start", b.start[1:]), ("block_table", b.table.long())):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_kv_attend_shared(**dict(good, **{name: bad}))
        assert e.value.code == moe.MOE_ERR_ARG
