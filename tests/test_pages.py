"""Shared pages (moe_kv_fork, moe_kv_reclaim, moe_kv_copy) against plain loops; all results are exact."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__

    __graft_entry__.build()
    import mxfp4_weight_mxfp8_gb300 as moe

    return moe


# ------------------------------------------------------------- plain references
def fork_reference(parents, table, lens, page, free, head):
    width, n = table.shape[1], len(parents)
    out, out_lens, moves = np.full((n, width), -1, np.int32), np.zeros(n, np.int32), np.tile(np.int32([-1, -1, 0]), (n, 1))
    seen, errors = set(), 0
    for r, p in enumerate(parents):
        if p == -1:
            continue
        if not 0 <= p < len(table):
            errors |= 1
            continue
        c = int(lens[p])
        if c < 0:
            errors |= 1
            c = 0
        out_lens[r] = c
        needed = -(-c // page)
        errors |= 4 if needed > width else 0
        out[r, :needed] = table[p, :needed]
        if p in seen and c % page and needed <= width and table[p, needed - 1] >= 0:
            if 0 <= head < len(free):
                out[r, needed - 1] = free[head]
                if free[head] >= 0:
                    moves[r] = table[p, needed - 1], free[head], c % page
            else:
                out[r, needed - 1] = -1
                errors |= 8
            head += 1
        seen.add(p)
    return out, out_lens, moves, [int((moves[:, 2] > 0).sum()), head, int(out_lens.max(initial=0)), errors]


def reclaim_reference(table, lens, page, pages, compact):
    held, errors, covered = set(), 0, []
    for row, c in zip(table, lens):
        errors |= 1 if c < 0 else 0
        n = -(-max(int(c), 0) // page)
        errors |= 4 if n > len(row) else 0
        covered.append(min(n, len(row)))
        for p in row[:covered[-1]]:
            if 0 <= p < pages:
                held.add(int(p))
            else:
                errors |= 2
    n = len(held)
    if not compact:
        return [p for p in range(pages) if p not in held], [n, n, 0, errors]
    leaves, places = sorted(p for p in held if p >= n), [p for p in range(n) if p not in held]
    to = dict(zip(leaves, places))
    out = np.full(table.shape, -1, np.int32)
    for r, c in enumerate(covered):
        for j in range(c):
            p = int(table[r, j])
            out[r, j] = to.get(p, p) if 0 <= p < pages else -1
    return list(range(n, pages)), [n, n, len(leaves), errors], out, [[p, to[p], page] for p in leaves]


def ints(v, dtype=torch.int32):
    return torch.as_tensor(np.asarray(v), dtype=dtype).cuda().contiguous()


def run_fork(moe, parents, table, lens, page, free, head, stride=None):
    n, width = len(parents), table.shape[1]
    t = ints(table)
    if stride:
        wide = torch.full((len(table), width + stride), -9, dtype=torch.int32, device="cuda")
        wide[:, :width] = t
        t = wide[:, :width]
    out = torch.full((n, width + (stride or 0)), -7, dtype=torch.int32, device="cuda")[:, :width]
    out_lens, moves, counts = ints([0] * n), torch.full((n, 3), -7, dtype=torch.int32, device="cuda"), ints([0] * 4)
    moe.moe_kv_fork(ints(parents), t, ints(lens), page, ints(free), ints([head]), out, out_lens, moves, counts)
    return [x.cpu().numpy() for x in (out, out_lens, moves)] + [counts.tolist()]


def check_fork(moe, *args, **kw):
    got, want = run_fork(moe, *args, **kw), fork_reference(*args)
    for g, w in zip(got[:3], want[:3]):
        assert (g == w).all()
    assert got[3] == want[3]
    return got


def random_tables(rng, rows, page, most, pages, shared=0.3):
    lens = np.array([int(rng.integers(0, most + 1)) for _ in range(rows)])
    width = max(1, -(-int(lens.max()) // page)) + 1
    table = np.full((rows, width), -1, np.int32)
    at, ids = 0, rng.permutation(pages)
    for r in range(rows):
        n = -(-int(lens[r]) // page)
        keep = 0
        if r and rng.random() < shared:
            keep = int(rng.integers(0, 1 + min(n, -(-int(lens[r - 1]) // page))))
            table[r, :keep] = table[r - 1, :keep]
        table[r, keep:n] = ids[at:at + n - keep]
        at += n - keep
        table[r, n:] = rng.integers(-1, pages, width - n)  # stale entries
    return table, lens, ids[at:]


# ------------------------------------------------------------------- refusals
def fork_block(moe, **changes):
    b = moe._KvFork(parents=0x1000, block_table=0x10000, table_stride=8, seq_lens=0x2000, free_pages=0x3000, free_head=0x4000,
                    out_table=0x20000, out_stride=8, out_lens=0x5000, moves=0x6000, counts=0x7000, rows=3, requests=4,
                    page_tokens=16, table_width=8, free_count=5)
    for k, v in changes.items():
        setattr(b, k, v)
    return b


@pytest.mark.parametrize("changes", [
    dict(requests=0), dict(requests=1025), dict(rows=0), dict(rows=1025), dict(page_tokens=17), dict(free_count=-1), dict(table_width=0),
    dict(table_width=2 ** 31 - 1, table_stride=2 ** 31, out_stride=2 ** 31),
    dict(table_stride=7), dict(out_stride=7), dict(parents=0), dict(block_table=0), dict(seq_lens=0), dict(free_pages=0), dict(free_head=0),
    dict(out_table=0), dict(out_lens=0), dict(moves=0), dict(counts=0), dict(parents=0x1002), dict(out_table=0x20001),
    dict(out_table=0x10000), dict(out_table=0x10020), dict(out_lens=0x2008), dict(counts=0x4000 - 12), dict(moves=0x5004), dict(counts=0x6010)])
def test_fork_refusals(moe, changes):
    assert moe.library().moe_kv_fork(ctypes.byref(fork_block(moe, **changes)), None) == moe.MOE_ERR_ARG
    assert moe.moe_last_error_detail()


def reclaim_block(moe, **changes):
    b = moe._KvReclaim(block_table=0x10000, table_stride=8, seq_lens=0x2000, free_pages=0x3000, counts=0x4000, out_table=0x20000, out_stride=8,
                       moves=0x30000, workspace=0x40000, requests=4, page_tokens=16, table_width=8, pages=100)
    for k, v in changes.items():
        setattr(b, k, v)
    return b


@pytest.mark.parametrize("changes", [
    dict(requests=0), dict(requests=1025), dict(page_tokens=8), dict(pages=0), dict(pages=(1 << 30) + 1), dict(table_width=0), dict(table_stride=4),
    dict(table_width=2 ** 31 - 1, table_stride=2 ** 31, out_table=0, moves=0, block_table=0x100000, free_pages=0x1000, seq_lens=0x900),
    dict(out_stride=7), dict(out_table=0), dict(moves=0), dict(block_table=0), dict(seq_lens=0), dict(free_pages=0), dict(counts=0),
    dict(workspace=0), dict(workspace=0x40008), dict(counts=0x4002), dict(free_pages=0x2000), dict(out_table=0x10004), dict(counts=0x3004),
    dict(out_table=0x10000, out_stride=9), dict(moves=0x10010), dict(workspace=0x30100)])
def test_reclaim_refusals(moe, changes):
    assert moe.library().moe_kv_reclaim(ctypes.byref(reclaim_block(moe, **changes)), None) == moe.MOE_ERR_ARG
    assert moe.moe_last_error_detail()


@pytest.mark.parametrize("changes", [dict(k=0), dict(k=0x10008), dict(pages=0), dict(page_tokens=48), dict(head_dim=96), dict(moves=0),
                                     dict(moves=0x3002), dict(count=0x4001), dict(capacity=-1)])
def test_copy_refusals(moe, changes):
    args = dict(moves=0x3000, count=None, capacity=2)
    c = moe._KvCache(k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x40000, pages=4, page_tokens=16, kv_heads=2, head_dim=64)
    for k, v in changes.items():
        if k in args:
            args[k] = v or None
        else:
            setattr(c, k, v)
    if "capacity" in changes:
        args["capacity"] = changes["capacity"]
    assert moe.library().moe_kv_copy(ctypes.byref(c), args["moves"], args["count"], args["capacity"], None) == moe.MOE_ERR_ARG


def test_null_blocks_and_no_moves(moe):
    assert moe.library().moe_kv_fork(None, None) == moe.MOE_ERR_ARG and moe.library().moe_kv_reclaim(None, None) == moe.MOE_ERR_ARG
    c = moe._KvCache(k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x40000, pages=4, page_tokens=16, kv_heads=2, head_dim=64)
    assert moe.library().moe_kv_copy(ctypes.byref(c), None, None, 0, None) == moe.MOE_OK


# ------------------------------------------------------------------------ fork
@pytest.mark.gpu
@pytest.mark.parametrize("rows,requests,page,most", [(1, 1, 16, 1), (1, 64, 64, 500), (8, 64, 128, 4000), (64, 64, 16, 3000), (257, 300, 32, 90),
                                                     (1000, 1024, 16, 2500), (1024, 1, 64, 64), (3, 256, 16, 0)])
def test_fork_matches_reference(moe, rows, requests, page, most):
    rng = np.random.default_rng(rows + requests)
    pages = rows * (most // page + 2) + requests + 9
    table, lens, free = random_tables(rng, rows, page, most, pages)
    parents = rng.integers(-1, rows, requests)
    check_fork(moe, parents, table, lens, page, free, 3)
    check_fork(moe, np.sort(parents), table, lens, page, free, 0, stride=5)


@pytest.mark.gpu
def test_fork_reports_what_does_not_fit(moe):
    table = np.int32([[0, 1, 2], [3, -1, 5], [6, 7, 8], [9, 10, 11]])
    lens = [40, 33, 500, -3]  # of row width 3 * 16: one too long, one negative
    parents = [0, 0, 0, 1, 1, 2, 2, 3, 3, 4, -2, -1, 2 ** 31 - 1]
    got = check_fork(moe, parents, table, lens, 16, [20, 21], 0)
    assert got[3][3] == 13  # three requests take a page (two of row 0, one of row 1), two are free
    got = check_fork(moe, parents, table, lens, 16, [20], 0)
    assert got[3][3] == 13 and (got[2][2] == [-1, -1, 0]).all()
    check_fork(moe, [0, 0], table, lens, 16, [], 0)
    check_fork(moe, [0, 0], table, lens, 16, [20, 21], -1)
    check_fork(moe, [0, 0], table, lens, 16, [20, 21], 2)
    check_fork(moe, [0, 0, 0], table, lens, 16, [-1, 21], 0)  # an empty place of the list
    check_fork(moe, [0, 0], table, [2 ** 31 - 1, 1, 1, 1], 128, [20], 0)


# ------------------------------------------------------------------------ copy
def make_cache(pages, heads, page, dim, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return tuple(torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)
                 for s in ((pages, heads, page, dim), (pages, heads, page, dim), (pages, heads), (pages, heads)))


def copy_reference(cache, moves):
    out = [c.clone() for c in cache]
    pages, page = cache[0].shape[0], cache[0].shape[2]
    for source, to, tokens in moves:
        if 0 <= source < pages and 0 <= to < pages and source != to and tokens > 0:
            for i in (0, 1):
                out[i][to, :, :min(tokens, page)] = cache[i][source, :, :min(tokens, page)]
            for i in (2, 3):
                out[i][to] = cache[i][source]
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("page,dim,heads", [(16, 64, 1), (16, 64, 3), (64, 128, 8), (128, 256, 2), (32, 128, 5)])
@pytest.mark.parametrize("n", [1, 7, 900])
def test_copy_matches_reference(moe, page, dim, heads, n):
    pages = 2 * n + 3
    cache = make_cache(pages, heads, page, dim, n)
    order = torch.randperm(pages).tolist()
    rng = np.random.default_rng(n)
    moves = [[order[i], order[n + i], int(rng.integers(1, page + 1))] for i in range(n)]
    moves += [[-1, -1, 0], [order[-1], order[-1], page], [pages, order[-1], 5], [order[-1], pages, 5], [order[-2], order[-1], 0],
              [order[-2], order[-1], -4], [-1, order[-1], page], [order[-2], -3, page], [2 ** 31 - 1, 0, 1]]
    moves[0][2] = page + 1000
    want = copy_reference(cache, moves)
    moe.moe_kv_copy(cache, ints(moves))
    assert all(torch.equal(c, w) for c, w in zip(cache, want))


@pytest.mark.gpu
@pytest.mark.parametrize("count", [-1, 0, 3, 5, 100])
def test_copy_stops_at_the_count(moe, count):
    cache = make_cache(12, 2, 16, 64, 1)
    moves = [[i, 6 + i, 16] for i in range(5)]
    want = copy_reference(cache, moves[:max(count, 0)])
    moe.moe_kv_copy(cache, ints(moves), ints([count]))
    assert all(torch.equal(c, w) for c, w in zip(cache, want))


@pytest.mark.gpu
def test_copy_past_32_bits(moe):
    """Pages beyond 4 GiB of a cache."""
    pages = (1 << 32) // (8 * 128 * 256) + 40
    k, v = (torch.zeros(pages, 8, 128, 256, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales = [torch.arange(pages * 8, device="cuda").view(pages, 8).to(torch.uint8) for _ in range(2)]
    k[pages - 2], v[pages - 2] = 3, 4
    moe.moe_kv_copy((k, v, *scales), ints([[pages - 2, pages - 1, 100], [0, pages - 3, 128]]))
    assert (k[pages - 1, :, :100] == 3).all() and (v[pages - 1, :, :100] == 4).all() and not k[pages - 1, :, 100:].any()
    assert torch.equal(scales[0][pages - 1], scales[0][pages - 2]) and torch.equal(scales[1][pages - 3], scales[1][0])
    assert not k[pages - 3].any() and (k[pages - 2] == 3).all()


# --------------------------------------------------------------------- reclaim
def run_reclaim(moe, table, lens, page, pages, compact, in_place=False, stride=0):
    width = table.shape[1]
    wide = torch.full((len(table), width + stride), -9, dtype=torch.int32, device="cuda")
    t = wide[:, :width]
    t.copy_(ints(table))
    free, counts = torch.full((pages,), -7, dtype=torch.int32, device="cuda"), ints([0] * 4)
    workspace = torch.full((moe.moe_kv_reclaim_bytes(pages) + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    out = moves = None
    if compact:
        out = t if in_place else torch.full_like(t, -8)
        moves = torch.full((max(1, pages // 2), 3), -7, dtype=torch.int32, device="cuda")
    moe.moe_kv_reclaim(t, ints(lens), page, free, counts, workspace, out, moves)
    assert (workspace[moe.moe_kv_reclaim_bytes(pages):] == 0xA5).all() and (wide[:, width:] == -9).all()
    return free.tolist(), counts.tolist(), None if out is None else out.cpu().numpy(), None if moves is None else moves.tolist()


def check_reclaim(moe, table, lens, page, pages, **kw):
    free, counts = reclaim_reference(table, lens, page, pages, False)
    got = run_reclaim(moe, table, lens, page, pages, False, **kw)
    n = counts[0]
    assert got[0] == [-7] * n + free and got[1] == counts
    for in_place in (False, True):
        free, counts, out, moves = reclaim_reference(table, lens, page, pages, True)
        got = run_reclaim(moe, table, lens, page, pages, True, in_place, **kw)
        assert got[0] == [-7] * n + free and got[1] == counts
        assert (got[2] == out).all()
        assert got[3][:len(moves)] == moves and all(m == [-7] * 3 for m in got[3][len(moves):])


@pytest.mark.gpu
@pytest.mark.parametrize("rows,page,most,spare", [(1, 16, 0, 0), (1, 16, 1, 0), (1, 64, 1, 1), (3, 64, 900, 5), (64, 64, 4000, 3000), (200, 32, 100, 31),
                                                  (1024, 16, 2000, 70000), (5, 128, 100000, 200000), (1000, 128, 1, 0)])
def test_reclaim_matches_reference(moe, rows, page, most, spare):
    rng = np.random.default_rng(rows + most)
    table, lens, _ = random_tables(rng, rows, page, most, rows * (most // page + 1) + spare)
    pages = rows * (most // page + 1) + spare
    lens[rng.random(rows) < 0.2] = 0
    check_reclaim(moe, table, lens, page, pages)
    check_reclaim(moe, table, lens, page, pages, stride=3)


@pytest.mark.gpu
@pytest.mark.parametrize("pages", [1, 2, 31, 32, 33, 64, 1023, 1024, 1025, 8192])
def test_reclaim_pools_that_are_empty_full_and_between(moe, pages):
    for held in {0, 1, pages // 2, max(pages - 1, 1), pages}:
        ids = np.random.default_rng(held).permutation(pages)[:held]
        table = np.full((1, max(held, 1)), -1, np.int32)
        table[0, :held] = ids
        check_reclaim(moe, table, [16 * held], 16, pages)


@pytest.mark.gpu
def test_reclaim_reports_bad_rows(moe):
    table = np.int32([[0, 1, 2, 3], [4, -1, 100, 7], [8, 9, 10, 11], [12, 13, 14, 15], [2, 2, 2, 40]])
    check_reclaim(moe, table, [64, 64, -5, 1000, 49], 16, 50)
    check_reclaim(moe, table, [64, 64, 0, 17, 64], 16, 50)
    check_reclaim(moe, table, [2 ** 31 - 1, 0, 0, 0, 0], 128, 50)


@pytest.mark.gpu
def test_a_pool_through_plans_forks_ends_and_compactions(moe):
    """Requests grow, fork, end and are compacted, in one run on the GPU; every request's tokens stay what they were."""
    rng = np.random.default_rng(5)
    page, width, pages, heads, dim = 16, 12, 60, 2, 64
    cache = moe.KvCache(pages, heads, page, dim)
    table = torch.full((6, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(6, dtype=torch.int32, device="cuda")
    free, head = torch.arange(pages, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    text = [[] for _ in range(6)]  # each request's tokens: a number that its keys hold in every element
    workspace = torch.zeros(moe.moe_kv_reclaim_bytes(pages), dtype=torch.uint8, device="cuda")
    for step in range(30):
        new = [int(rng.integers(0, 9)) if len(t) < 120 else 0 for t in text]
        total = sum(new)
        q_start, seq, counts = torch.empty(7, dtype=torch.int32, device="cuda"), torch.empty_like(lens), torch.empty(4, dtype=torch.int32, device="cuda")
        positions, slots = torch.empty(total, dtype=torch.int32, device="cuda"), torch.empty(total, dtype=torch.int64, device="cuda")
        moe.moe_kv_plan(lens, ints(new), page, table, free, head, q_start, seq, positions, slots, counts)
        lens, head = seq, counts[1:2]
        said = [2.0 ** float(v) for v in rng.integers(-3, 4, total)]
        at = 0
        for t, n in zip(text, new):
            t += said[at:at + n]
            at += n
        rows = torch.tensor(said, device="cuda").to(torch.bfloat16)[:, None, None].expand(total, heads, dim)
        if total:
            cache.append(rows.contiguous(), (-rows).contiguous(), slots)
        assert counts[3].item() == 0
        if step % 3 == 1:  # samples and reordered rows
            parents = [int(v) for v in rng.integers(-1, 6, 6)]
            out, out_lens, moves, c = torch.empty_like(table), torch.empty_like(lens), ints([[0] * 3] * 6), torch.empty_like(counts)
            moe.moe_kv_fork(ints(parents), table, lens, page, free, head, out, out_lens, moves, c)
            cache.copy(moves)
            table, lens, head = out, out_lens, c[1:2]
            text = [list(text[p]) if p >= 0 else [] for p in parents]
            assert c[3].item() == 0
        if step % 4 == 2:  # a request ends; every other time the pool is compacted
            lens = lens.clone()
            lens[step % 6] = 0
            text[step % 6] = []
            compact = step % 8 == 2
            free, c = torch.empty(pages, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
            moves = torch.empty(pages // 2, 3, dtype=torch.int32, device="cuda") if compact else None
            moe.moe_kv_reclaim(table, lens, page, free, c, workspace, table if compact else None, moves)
            if compact:
                cache.copy(moves, c[2:3])
                held = {int(p) for r in range(6) for p in table[r, : -(-len(text[r]) // page)].tolist()}
                assert held == set(range(c[0].item()))
            head = c[1:2]
            assert c[3].item() == 0
        for r, t in enumerate(text):
            assert lens[r].item() == len(t)
            for i, want in enumerate(t):
                p = table[r, i // page].item()
                key = cache.k.view(torch.float8_e4m3fn)[p, :, i % page].float() * torch.exp2(cache.k_scale[p].float() - 127)[:, None]
                value = cache.v.view(torch.float8_e4m3fn)[p, :, i % page].float() * torch.exp2(cache.v_scale[p].float() - 127)[:, None]
                assert (key == want).all() and (value == -want).all(), (step, r, i)


@pytest.mark.gpu
def test_fork_reclaim_and_copy_in_a_graph(moe):
    rng = np.random.default_rng(8)
    table, lens, free = random_tables(rng, 20, 16, 300, 500)
    cache = make_cache(500, 2, 16, 64, 3)
    t, l, p = ints(table), ints(lens), ints(rng.integers(0, 20, 30))
    out, out_lens, moves, counts = torch.empty(30, table.shape[1], dtype=torch.int32, device="cuda"), ints([0] * 30), ints([[0] * 3] * 30), ints([0] * 4)
    f, h = ints(free), ints([0])
    rf, rc = torch.zeros(500, dtype=torch.int32, device="cuda"), ints([0] * 4)
    workspace = torch.zeros(moe.moe_kv_reclaim_bytes(500), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_kv_fork(p, t, l, 16, f, h, out, out_lens, moves, counts)
        moe.moe_kv_copy(cache, moves)
        moe.moe_kv_reclaim(out, out_lens, 16, rf, rc, workspace)
    for seed in (1, 2):
        parents = np.random.default_rng(seed).integers(-1, 20, 30)
        p.copy_(ints(parents))
        before = [c.clone() for c in cache]
        graph.replay()
        want = fork_reference(parents, table, lens, 16, free, 0)
        assert (out.cpu().numpy() == want[0]).all() and counts.tolist() == want[3]
        assert all(torch.equal(c, w) for c, w in zip(cache, copy_reference(before, want[2].tolist())))
        listed, rcounts = reclaim_reference(want[0], want[1], 16, 500, False)
        assert rc.tolist() == rcounts and rf.tolist()[rcounts[0]:] == listed


@pytest.mark.gpu
def test_pages_python_refusals(moe):
    table, lens, one = ints([[0, 1]]), ints([20]), ints([0])
    free, counts, moves = ints([2, 3]), ints([0] * 4), ints([[0] * 3])
    w = torch.zeros(moe.moe_kv_reclaim_bytes(2), dtype=torch.uint8, device="cuda")
    cache = make_cache(4, 1, 16, 64, 0)
    bad = [lambda: moe.moe_kv_fork(one, table, lens, 16, free, one, table, lens.clone(), moves, counts),
           lambda: moe.moe_kv_fork(one, table, lens, 16, free, one, ints([[0, 0, 0]]), lens.clone(), moves, counts),
           lambda: moe.moe_kv_fork(one, table, lens, 16, free, one, table.clone(), lens.clone(), moves[:, :2], counts),
           lambda: moe.moe_kv_fork(one.cpu(), table, lens, 16, free, one, table.clone(), lens.clone(), moves, counts),
           lambda: moe.moe_kv_fork(one, table.cpu(), lens, 16, free, one, table.clone(), lens.clone(), moves, counts),
           lambda: moe.moe_kv_reclaim(table, lens, 16, free, counts, w[:-1]), lambda: moe.moe_kv_reclaim(table, lens, 16, free, counts, w, table.clone()),
           lambda: moe.moe_kv_reclaim(table, lens, 16, ints([0] * 8), counts, torch.zeros(2000, dtype=torch.uint8, device="cuda"), table.clone(), moves),
           lambda: moe.moe_kv_copy(cache, moves[:, :2]), lambda: moe.moe_kv_copy(cache, moves.long()), lambda: moe.moe_kv_copy(cache, moves, counts),
           lambda: moe.moe_kv_copy(cache[:2] + cache[:2], moves)]
    for call in bad:
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.code == moe.MOE_ERR_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("before", ["nothing", "memcpy", "memset", "join"])
def test_copy_in_a_graph_behind_what_is_no_kernel(moe, before):
    """Its launch is a chained one; the moves come by a memcpy, or from another stream."""
    cache = [torch.randint(0, 255, s, dtype=torch.uint8, device="cuda") for s in ((9, 2, 16, 64), (9, 2, 16, 64), (9, 2), (9, 2))]
    source = torch.tensor([[0, 4, 16], [1, 5, 7], [-1, -1, 0]], dtype=torch.int32, device="cuda")
    moves = source.clone() if before in ("nothing", "memset") else torch.zeros_like(source)
    junk, other, graph = torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    want = [c.clone() for c in cache]
    for c, w in zip(cache, want):
        w[4], w[5] = c[0], c[1]
        if c.dim() == 4:
            w[5][:, 7:] = c[5][:, 7:]
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        if before == "memcpy":
            moves.copy_(source)
        elif before == "memset":
            junk.zero_()
        elif before == "join":
            other.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(other):
                moves.copy_(source)
            junk.fill_(3)
            torch.cuda.current_stream().wait_stream(other)
        moe.moe_kv_copy(tuple(cache), moves)
    graph.replay()
    torch.cuda.synchronize()
    for c, w in zip(cache, want):
        assert torch.equal(c, w)
