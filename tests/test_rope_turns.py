"""moe_rope_turns against the formula in 80 digits: the table is its values rounded to units of 2^-64 turns.

Angles of far positions are the table's entries times up to 2^31, so a table of
a double's 53 bits would be 2^-25 of a turn off there.
"""
from __future__ import annotations

from decimal import ROUND_CEILING, ROUND_FLOOR, Decimal, getcontext

import numpy as np
import pytest
import torch
from test_rope import check, moe  # noqa: F401

TAU = Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257241799725606965068423413596")


def table(n, base, scaling, factor, trained, low, high):
    getcontext().prec = 80
    base, factor, trained, low, high = (Decimal(float(x)) for x in (base, factor, trained, low, high))

    def index(turns):
        return n * (trained / (TAU * turns)).ln() / (2 * base.ln())

    a = max(index(high).to_integral_value(ROUND_FLOOR), Decimal(0))
    b = min(index(low).to_integral_value(ROUND_CEILING), Decimal(n - 1))
    out = []
    for i in range(n // 2):
        f, s = base ** (Decimal(-2 * i) / n), Decimal(0)
        if scaling == 1:
            s = (trained * f / TAU - low) / (high - low)
        elif scaling == 2:
            s = 1 - (i - a) / (b - a if b > a else Decimal("0.001"))
        s = min(max(s, Decimal(0)), Decimal(1))
        f = f * s + f / factor * (1 - s)
        out.append(int((f / TAU * 2 ** 64).to_integral_value()) % 2 ** 64)
    return out


@pytest.mark.parametrize("n", [2, 6, 24, 64, 128, 512])
@pytest.mark.parametrize("base,scaling,factor,trained,low,high", [
    (1e4, 0, 1.0, 8192, 1, 4), (5e5, 0, 4.0, 8192, 1, 4), (1e6, 1, 8.0, 8192, 1, 4), (1e4, 2, 32.0, 4096, 1, 32), (700.0, 2, 4.0, 8192, 1, 4),
    (1e4, 0, 0.05, 8192, 1, 4), (1.5, 2, 2.0, 8192, 1, 4), (1.0000001, 0, 3.0, 8192, 1, 4), (1e300, 1, 0.3, 131072, 0.5, 7), (12345.678, 2, 1e-6, 100, 1, 4),
    (5e6, 1, 16.0, 32768, 1, 32)])
def test_turns_are_the_formulas_rounded_once(moe, n, base, scaling, factor, trained, low, high):  # noqa: F811
    got = [v % 2 ** 64 for v in moe.moe_rope_turns(n, base, scaling, factor, trained, low, high).tolist()]
    assert got == table(n, base, scaling, factor, trained, low, high)


@pytest.mark.gpu
@pytest.mark.parametrize("base", [1e4, 1e6])
def test_far_positions_turn_by_the_formula_itself(moe, base):  # noqa: F811
    """The angle of position 2^31 - 1 in 80 digits, not from the table."""
    n, positions = 128, [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 1]
    turns = moe.moe_rope_turns(n, base, device="cuda")
    getcontext().prec = 80
    angles = np.array([[float((p * Decimal(base) ** (Decimal(-2 * i) / n) / TAU) % 1 * TAU) for i in range(n // 2)] for p in positions])
    angle = torch.from_numpy(angles).cuda()[:, None]
    q = torch.randn(len(positions), 3, n, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    moe.moe_rope(torch.tensor(positions, dtype=torch.int32, device="cuda"), turns, q, q_out=out)
    a, b = q.double()[..., :n // 2], q.double()[..., n // 2:]
    want = torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1)
    size = (a.abs() + b.abs()).repeat(1, 1, 2)
    # Half a unit of the table is 2^-34 of a turn at 2^31, what the angle drops 2^-32: under 2e-9; the rest as in test_rope.
    check(out, want, size)
