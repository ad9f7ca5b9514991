"""Numbers that the C entries have no room for are refused as their other arguments are, natively and by the package's checks."""
from __future__ import annotations

import pytest
import torch
from test_shared import Batch, moe, same  # noqa: F401

HUGE = (2 ** 31, 2 ** 32 + 16, 2 ** 70)


@pytest.mark.parametrize("n", HUGE + (-1, -2 ** 32 + 64, -2 ** 32 + 2, -2 ** 70))
def test_sizes_on_the_host(moe, n):  # noqa: F811
    for args in ((n, 8, 64), (1, n, 64), (1, 8, n)):
        assert moe.moe_kv_shared_bytes(*args) == 0
    for args in ((n,), (64, 1e4, n)):  # (a table of one entry is no room for that of n modulo 2^32)
        with pytest.raises(moe.MoeError) as e:
            moe.moe_rope_turns(*args)
        assert e.value.code == moe.MOE_ERR_ARG


def refused(moe, call):  # noqa: F811
    for stream in (None, torch.cuda.current_stream()):
        with pytest.raises(moe.MoeError) as e:
            call(stream)
        assert e.value.code == moe.MOE_ERR_ARG


@pytest.mark.gpu
def test_numbers_past_their_fields(moe):  # noqa: F811
    b = Batch(moe, [(200, same(5, 30))], 64, 2, 128, 8, seed=12, pad=0)
    out = torch.empty(b.q.shape, dtype=torch.bfloat16, device="cuda")
    scratch = torch.empty(moe.moe_kv_shared_bytes(*b.q.shape), dtype=torch.uint8, device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    x, w = torch.zeros(2, 64, device="cuda"), torch.zeros(64, device="cuda")
    q = torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    room = torch.zeros(moe.moe_kv_reclaim_bytes(8), dtype=torch.uint8, device="cuda")
    for cache in (tuple(b.cache), list(b.cache)):
        for n in HUGE:
            refused(moe, lambda s: moe.moe_kv_attend_shared(cache, b.q, b.table, b.start, b.lens, b.group_start, b.prefix_lens, out, b.workspace,
                                                            scratch, least_tiles=n, stream=s))
    for n in HUGE:
        refused(moe, lambda s: moe.moe_kv_fork(i(3), i(3, 4), i(3), n, i(8), i(1), i(3, 4), i(3), i(3, 3), i(4), stream=s))
        refused(moe, lambda s: moe.moe_kv_reclaim(i(3, 4), i(3), n, i(8), i(4), room, stream=s))
    for value in (1e39, float("inf"), float("nan")):
        refused(moe, lambda s: moe.moe_norm(x, w, x, value, stream=s))
        refused(moe, lambda s: moe.moe_norm(x, w, x, weight_offset=value, stream=s))
        refused(moe, lambda s: moe.moe_rope(i(2), moe.moe_rope_turns(64, device="cuda"), q, amplitude=value, stream=s))


@pytest.mark.gpu
def test_cache_calls_refuse_queries_of_other_shapes(moe):  # noqa: F811
    c, i = moe.KvCache(4, 2, 16, 64), lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    q, table = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    for bad in (q[0], q[None], q[..., :32], q.float(), q.cpu()):
        with pytest.raises(moe.MoeError) as e:
            c.attend_shared(bad, table, i(0, 1, 2), i(1, 1), i(0, 2), i(16))
        assert e.value.code == moe.MOE_ERR_ARG
