"""moe_kv_attend, the form of many query rows: weights keep their precision when a reference is raised inside a tile.

Tolerance, derived before its first run: weights are held within 2^-16 of
themselves, queries within 2^-21 of their row's largest element, sums are FP32:
less than 2^-12 of sum_j w_j |v_j|; the output is rounded to BF16 once, 2^-8 of
it. (A weight rounded to BF16 alone would be 2^-9 off.)
"""
from __future__ import annotations

import numpy as np
import pytest
import torch
from test_decode_step import attend_reference, bf16, e4m3_encode, make_batch, moe, run_attend  # noqa: F401


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("at", [20, 50, 100])
@pytest.mark.parametrize("gap", [6.0, 9.0])
def test_weights_under_a_reference_raised_inside_a_tile(moe, gap, at, dim):  # noqa: F811
    """In two tiles four tokens carry all of the values; a later token of each tile, `gap` nats above them, has none.

    The one head is given many times over: then a CTA takes several tiles of it, the later ones against the first ones'
    references. (A tile that starts a CTA's run takes its own.)
    """
    rng = np.random.default_rng(dim + at)
    rows, q_heads, tokens = 60, 4, 900
    cache, table, start, seq = make_batch(rng, [(tokens, rows)], 64, 1, dim)
    k, v, ks, vs = cache
    ks[:], vs[:] = 120, 120
    v[:] = 0
    direction = np.where(rng.random(dim) < 0.5, -1.0, 1.0)
    q = bf16(np.broadcast_to(direction, (rows, q_heads, dim)) * (1 + 0.2 * rng.random((rows, q_heads, 1))))
    nats = np.full(tokens, -40.0)
    for base in (512, 640):
        few = base + np.array([1, 5, 9, 14])
        nats[few] = rng.uniform(-1, 1, 4)
        nats[base + at] = gap
        v[table[0, few // 64], 0, few % 64] = e4m3_encode(rng.standard_normal((4, dim)) * 60)
    for j in range(tokens):
        k[table[0, j // 64], 0, j % 64] = e4m3_encode(direction * nats[j] * dim ** -0.5 * 2.0 ** 7)
    heads = 64
    many = [np.repeat(c, heads, axis=1) for c in cache]
    out, _ = run_attend(moe, many, q.cuda().repeat(1, heads, 1), table, start, seq)
    exact, _, mass = attend_reference(cache, q.float().numpy(), table, start, seq, dim ** -0.5, 0)
    out = out.reshape(rows, heads, q_heads, dim)
    assert (np.abs(out - exact[:, None]) <= (2.0 ** -8 * np.abs(exact) + 2.0 ** -12 * mass)[:, None]).all()
