"""moe_rope and moe_rope_turns against the formula with whole-number angles and 64 bits.

Tolerance, derived before its first run: the angle is exact to 2^-32 of a turn, its
conversion to FP32 half turns rounds to 2^-25 of one, sincospif is within 2 ulp:
together under 5e-7 in sine and cosine. Two products and a sum in FP32 add less
than 4 u; the output is half a step of BF16 (2^-8 relative) off.
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


# ----------------------------------------------------------------- on the host
def turns_reference(n, base, scaling, factor, trained, low, high):
    from fractions import Fraction

    out = []
    for i in range(n // 2):
        f = base ** (-2.0 * i / n)
        if scaling == 1:
            s = min(max((trained * f / math.tau - low) / (high - low), 0.0), 1.0)
        elif scaling == 2:
            at = lambda turns: n * math.log(trained / (math.tau * turns)) / (2 * math.log(base))  # noqa: E731
            a, b = max(math.floor(at(high)), 0), min(math.ceil(at(low)), n - 1)
            s = 1.0 - min(max((i - a) / (b - a if b > a else 0.001), 0.0), 1.0)
        else:
            s = 0.0
        f = f * s + f / factor * (1 - s)
        out.append(round(Fraction(f) / Fraction(math.tau) * 2 ** 64) % 2 ** 64)
    return out


@pytest.mark.parametrize("n", [2, 6, 64, 128, 512])
@pytest.mark.parametrize("base,scaling,factor", [(1e4, 0, 1.0), (5e5, 0, 4.0), (1e6, 1, 8.0), (1e4, 2, 32.0), (700.0, 2, 4.0), (1e4, 0, 0.05), (1.5, 2, 2.0)])
def test_turns_match_the_formula(moe, n, base, scaling, factor):
    got = [v % 2 ** 64 for v in moe.moe_rope_turns(n, base, scaling, factor, 8192.0, 1.0, 4.0).tolist()]
    want = turns_reference(n, base, scaling, factor, 8192.0, 1.0, 4.0)
    for g, w in zip(got, want):  # a few roundings in 64 bits of a number below 2^64 (a sum of two, a power, a quotient)
        assert min((g - w) % 2 ** 64, (w - g) % 2 ** 64) <= 16 * 2.0 ** -53 * 2 ** 64 * max(1.0, 1 / factor)


def test_turns_of_a_whole_and_of_half_a_turn(moe):
    """A factor that makes the first pair turn once, or half, a position."""
    whole = moe.moe_rope_turns(2, 1e4, 0, 1 / math.tau)[0].item() % 2 ** 64
    assert min(whole, 2 ** 64 - whole) <= 2 ** 13
    half = moe.moe_rope_turns(2, 1e4, 0, 2 / math.tau)[0].item() % 2 ** 64
    assert abs(half - 2 ** 63) <= 2 ** 13


@pytest.mark.parametrize("args", [(0,), (3,), (514,), (8, 1.0), (8, float("inf")), (8, 1e4, 3), (8, 1e4, 0, 0.0), (8, 1e4, 0, float("nan")),
                                  (8, 1e4, 1, 2.0, 0.0), (8, 1e4, 1, 2.0, 8192.0, 0.0), (8, 1e4, 2, 2.0, 8192.0, 4.0, 4.0)])
def test_turns_refusals(moe, args):
    with pytest.raises(moe.MoeError) as e:
        moe.moe_rope_turns(*args)
    assert e.value.code == moe.MOE_ERR_ARG


def block(moe, **changes):
    b = moe._Rope(positions=0x1000, turns=0x2000, q=0x10000, q_token_stride=256, q_head_stride=64, q_out=0x20000, q_out_token_stride=256,
                  q_out_head_stride=64, k=0x30000, k_token_stride=128, k_head_stride=64, k_out=0x40000, k_out_token_stride=128,
                  k_out_head_stride=64, tokens=3, q_heads=4, k_heads=2, head_dim=64, rotary_dim=64, amplitude=1.0)
    for k, v in changes.items():
        setattr(b, k, v)
    return b


@pytest.mark.parametrize("changes", [
    dict(tokens=-1), dict(q_heads=0), dict(q_heads=1025), dict(k_heads=-1), dict(head_dim=1), dict(head_dim=514), dict(rotary_dim=0),
    dict(rotary_dim=63), dict(rotary_dim=66), dict(amplitude=float("nan")), dict(q_token_stride=-1), dict(k_out_head_stride=-64),
    dict(positions=0), dict(turns=0), dict(q=0), dict(q_out=0), dict(k=0), dict(k_out=0), dict(positions=0x1002), dict(turns=0x2004),
    dict(q=0x10001), dict(q_out=0x10000, q_out_head_stride=128, q_out_token_stride=512), dict(q_out=0x10002), dict(q_out_head_stride=32),
    dict(q_out_token_stride=128), dict(q_out_token_stride=0), dict(k_out=0x20000), dict(k_out=0x10000), dict(q_out=0x30000),
    dict(q_out=0x1000 - 0x400)])
def test_rope_refusals(moe, changes):
    assert moe.library().moe_rope(ctypes.byref(block(moe, **changes)), None) == moe.MOE_ERR_ARG
    assert moe.moe_last_error_detail()


def test_rope_of_no_tokens_is_no_work(moe):
    assert moe.library().moe_rope(ctypes.byref(block(moe, tokens=0, q=0)), None) == moe.MOE_OK
    assert moe.library().moe_rope(None, None) == moe.MOE_ERR_ARG


# --------------------------------------------------------------------- rotated
def rotate(x, positions, turns, interleaved, amplitude=1.0):
    """(rotated, |a| + |b| of each element's pair) in float64."""
    t = turns.cpu().numpy().view(np.uint64)
    with np.errstate(over="ignore"):
        whole = positions.cpu().numpy().astype(np.int64).view(np.uint64)[:, None] * t
    angle = torch.from_numpy(whole.astype(np.float64) * 2.0 ** -64 * math.tau).cuda()[:, None]
    y, size, n = x.double().clone(), torch.zeros_like(x, dtype=torch.float64), 2 * len(t)
    i = torch.arange(n // 2, device="cuda")
    a_at, b_at = (2 * i, 2 * i + 1) if interleaved else (i, i + n // 2)
    a, b = x.double()[..., a_at], x.double()[..., b_at]
    y[..., a_at] = amplitude * (a * torch.cos(angle) - b * torch.sin(angle))
    y[..., b_at] = amplitude * (b * torch.cos(angle) + a * torch.sin(angle))
    size[..., a_at] = size[..., b_at] = amplitude * (a.abs() + b.abs())
    return y, size


def check(got, want, size):
    err = (got.double() - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + 1e-6 * size + 2.0 ** -134).all()


CASES = [(1, 1, 1, 64, 64), (1, 64, 8, 128, 128), (5, 4, 4, 64, 32), (33, 28, 4, 128, 64), (700, 8, 1, 128, 128), (3, 5, 0, 256, 256), (2, 16, 2, 96, 96),
         (17, 3, 1, 96, 24), (9, 6, 2, 128, 2), (4, 2, 2, 80, 80), (6, 3, 3, 66, 30), (2, 1024, 1, 64, 64), (1, 2, 1, 512, 512), (2000, 4, 2, 64, 64),
         (2, 3, 2, 257, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,q_heads,k_heads,dim,rotary", CASES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_matches_64_bits(moe, tokens, q_heads, k_heads, dim, rotary, interleaved):
    g = torch.Generator(device="cuda").manual_seed(tokens + dim)
    # A projection's output: queries, keys and values side by side.
    qkv = torch.randn(tokens, q_heads + 2 * k_heads, dim, generator=g, device="cuda").to(torch.bfloat16)
    q, k = qkv[:, :q_heads], qkv[:, q_heads:q_heads + k_heads] if k_heads else None
    positions = torch.randint(0, 1 << 20, (tokens,), generator=g, device="cuda").int()
    positions[0] = 2 ** 31 - 1
    if tokens > 2:
        positions[1], positions[2] = 0, -5
    turns = moe.moe_rope_turns(rotary, 1e6, moe.ROPE_BANDS, 8.0, device="cuda")
    q_out = torch.full((tokens, q_heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((tokens, k_heads, dim), 7.0, dtype=torch.bfloat16, device="cuda") if k_heads else None
    before = qkv.clone()
    moe.moe_rope(positions, turns, q, k, q_out, k_out, interleaved=interleaved, amplitude=1.25)
    assert torch.equal(qkv, before)
    check(q_out, *rotate(q, positions, turns, interleaved, 1.25))
    assert torch.equal(q_out[..., rotary:], q[..., rotary:])
    if k_heads:
        check(k_out, *rotate(k, positions, turns, interleaved, 1.25))
        assert torch.equal(k_out[..., rotary:], k[..., rotary:])
    # In place, the values untouched, the same bits.
    moe.moe_rope(positions, turns, q, k, interleaved=interleaved, amplitude=1.25)
    assert torch.equal(q, q_out) and (k is None or torch.equal(k, k_out))
    assert torch.equal(qkv[:, q_heads + k_heads:], before[:, q_heads + k_heads:])
    # Head-major outputs, and rows that are not on 16-byte boundaries.
    turned = torch.zeros(q_heads, tokens, dim, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    odd = torch.zeros(tokens, q_heads, dim + 1, dtype=torch.bfloat16, device="cuda")[..., 1:]
    for out in (turned, odd):
        moe.moe_rope(positions, turns, before[:, :q_heads], q_out=out, interleaved=interleaved, amplitude=1.25)
        assert torch.equal(out, q_out)


@pytest.mark.gpu
def test_rope_far_positions_turn_as_near_ones(moe):
    """A pair that turns 2^-k of a turn a position is back after 2^k of them, exactly."""
    turns = torch.tensor([1 << 40, 1 << 50] * 8, dtype=torch.int64, device="cuda")
    x = torch.randn(2, 3, 32, device="cuda").to(torch.bfloat16)
    x[1] = x[0]
    out = torch.empty_like(x)
    moe.moe_rope(torch.tensor([77, 77 + (1 << 24)], dtype=torch.int32, device="cuda"), turns, x, q_out=out)
    assert torch.equal(out[0], out[1])


@pytest.mark.gpu
def test_rope_in_a_graph_and_on_a_stream(moe):
    turns = moe.moe_rope_turns(128, device="cuda")
    positions = torch.arange(64, dtype=torch.int32, device="cuda")
    q = torch.randn(64, 16, 128, device="cuda").to(torch.bfloat16)
    out, want = torch.empty_like(q), torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_rope(positions, turns, q, q_out=out)
    positions += 1000
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_rope(positions, turns, q, q_out=want, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    check(out, *rotate(q, positions, turns, False))


@pytest.mark.gpu
def test_rope_infinities_and_nan_stay_in_their_pair(moe):
    turns = moe.moe_rope_turns(64, device="cuda")
    q = torch.ones(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 3], q[0, 1, 40] = float("nan"), float("inf")
    out = torch.empty_like(q)
    moe.moe_rope(torch.tensor([5], dtype=torch.int32, device="cuda"), turns, q, q_out=out)
    bad = ~torch.isfinite(out[0])
    assert bad.nonzero().tolist() == [[0, 3], [0, 35], [1, 8], [1, 40]]


@pytest.mark.gpu
def test_rope_python_refusals(moe):
    turns = moe.moe_rope_turns(64, device="cuda")
    p = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: moe.moe_rope(p, turns, q.float()), lambda: moe.moe_rope(p, turns.cpu(), q), lambda: moe.moe_rope(p[:1], turns, q),
                lambda: moe.moe_rope(p, turns, q[..., :62]), lambda: moe.moe_rope(p, turns, q, q_out=q[:, :2]),
                lambda: moe.moe_rope(p, turns, q, k=q[:1]), lambda: moe.moe_rope(p, turns, q, k_out=q), lambda: moe.moe_rope(p.long(), turns, q),
                lambda: moe.moe_rope(p, turns, q.transpose(1, 2)), lambda: moe.moe_rope(p, turns, q, k=q)):
        with pytest.raises(moe.MoeError) as e:
            bad()
        assert e.value.code == moe.MOE_ERR_ARG
