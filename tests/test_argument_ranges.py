"""Numbers that the C entries have no room for are refused as their other arguments are."""
from __future__ import annotations

import pytest
from test_shared import moe  # noqa: F401

HUGE = (2 ** 31, 2 ** 32 + 16, 2 ** 70)


@pytest.mark.parametrize("n", HUGE + (-1, -2 ** 32 + 64, -2 ** 32 + 2, -2 ** 70))
def test_sizes_on_the_host(moe, n):  # noqa: F811
    for args in ((n, 8, 64), (1, n, 64), (1, 8, n)):
        assert moe.moe_kv_shared_bytes(*args) == 0
    for args in ((n,), (64, 1e4, n)):  # (a table of one entry is no room for that of n modulo 2^32)
        with pytest.raises(moe.MoeError) as e:
            moe.moe_rope_turns(*args)
        assert e.value.code == moe.MOE_ERR_ARG
