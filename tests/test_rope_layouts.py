"""moe_rope on queries and keys that lie between one another: taken in place wherever no byte is shared, and refused elsewhere."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch
from test_rope import check, moe, rotate  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Run where no GPU is to be seen: what the checks let pass ends as a failed launch, MOE_ERR_CUDA, and touches no memory.
ON_CPU = """
import ctypes, random, sys
import mxfp4_weight_mxfp8_gb300 as moe

def status(T, D, q, k, q_out=None, k_out=None):
    b = moe._Rope(positions=0x10, turns=0x200, tokens=T, q_heads=q[3], k_heads=k[3], head_dim=D, rotary_dim=D, amplitude=1.0)
    for name, (at, token, head, _) in (("q", q), ("q_out", q_out or q), ("k", k), ("k_out", k_out or k)):
        setattr(b, name, 0x1000000 + 2 * at), setattr(b, name + "_token_stride", token), setattr(b, name + "_head_stride", head)
    return moe.library().moe_rope(ctypes.byref(b), None)

def elements(T, D, x):
    at, token, head, heads = x
    return [at + t * token + h * head + i for t in range(T) for h in range(heads) for i in range(D)]

def expected(T, D, q, k, q_out, k_out):
    sets = [elements(T, D, x) for x in (q, k, q_out or q, k_out or k)]
    qi, ki, qo, ko = map(set, sets)
    if len(qo) < len(sets[2]) or len(ko) < len(sets[3]) or qo & ko or qo & ki or ko & qi:
        return False
    return not (q_out and qo & qi or k_out and ko & ki)

def exact(T, tensors):
    # Tensors of different token strides are only told apart by their ranges of memory.
    return T == 1 or len({x[1] for x in tensors}) == 1

rng = random.Random(5)
taken = refused = 0
for _ in range(6000):
    T, D = rng.choice([1, 1, 2, 3, 5]), 2 * rng.randint(1, 4)
    kind = rng.randrange(4)
    heads = rng.randint(1, 4)
    if kind == 0:    # [T, heads, parts, D]
        parts = rng.randint(2, 4)
        token, head, unit = heads * parts * D, parts * D, D
    elif kind == 1:  # [heads, parts, T, D]
        parts = rng.randint(2, 4)
        token, head, unit = D, parts * T * D, T * D
    elif kind == 2:  # [T, parts * heads, D]
        parts = rng.randint(2, 4)
        token, head, unit = parts * heads * D + rng.choice([0, 3]), D, heads * D
    else:            # any
        parts, token, head, unit = 3, rng.randint(0, 40), rng.randint(0, 30), rng.randint(1, 40)
    def one(i, other=False):
        step = 0 if rng.random() < 0.8 else rng.randint(-3, 3)
        return (200 + i * unit + step, token, head if kind < 3 or not other else rng.randint(0, 30), rng.randint(1, heads))
    q, k = one(0), one(rng.randrange(1, parts), True)
    out = rng.random() < 0.3
    q_out = (one(rng.randrange(parts))[:3] + (q[3],)) if out else None
    k_out = (one(rng.randrange(parts), True)[:3] + (k[3],)) if out and rng.random() < 0.5 else None
    if q_out and q_out[:3] == q[:3]: q_out = None
    if k_out and k_out[:3] == k[:3]: k_out = None
    want, got = expected(T, D, q, k, q_out, k_out), status(T, D, q, k, q_out, k_out)
    assert got in (moe.MOE_ERR_ARG, moe.MOE_ERR_CUDA), got
    assert (got == moe.MOE_ERR_CUDA) == want, (T, D, q, k, q_out, k_out, want, moe.moe_last_error_detail())
    taken, refused = taken + want, refused + (not want)
assert taken > 1000 and refused > 1000, (taken, refused)

# Of different token strides: never taken where a byte is shared, always in ranges of their own.
for _ in range(3000):
    T, D = rng.choice([2, 3, 5]), 2 * rng.randint(1, 4)
    q, k = [(200 + rng.randint(0, 300), rng.randint(0, 60), rng.randint(0, 30), rng.randint(1, 4)) for _ in range(2)]
    want, got = expected(T, D, q, k, None, None), status(T, D, q, k)
    if got == moe.MOE_ERR_CUDA:
        assert want, (T, D, q, k)
    a, b = elements(T, D, q), elements(T, D, k)
    if want and (max(a) < min(b) or max(b) < min(a)):
        assert got == moe.MOE_ERR_CUDA, (T, D, q, k)

# A fused projection [T, heads, 3, D], queries and keys turned where they lie.
for T in (1, 5, 70000):
    assert status(T, 64, (0, 1536, 192, 8), (64, 1536, 192, 8)) == moe.MOE_ERR_CUDA
    assert status(T, 64, (0, 1536, 192, 8), (63, 1536, 192, 8)) == moe.MOE_ERR_ARG
    assert status(T, 64, (0, 1536, 192, 8), (64, 1536, 192, 8), (128, 1536, 192, 8)) == moe.MOE_ERR_CUDA
    assert status(T, 64, (0, 1536, 192, 8), (64, 1536, 192, 8), (64, 1536, 192, 8)) == moe.MOE_ERR_ARG
print("done", taken, refused)
"""


def test_layouts_are_taken_where_no_byte_is_shared_and_refused_elsewhere(moe):  # noqa: F811
    run = subprocess.run([sys.executable, "-c", ON_CPU], cwd=ROOT, env=dict(os.environ, CUDA_VISIBLE_DEVICES="-1"), capture_output=True, text=True)
    assert run.returncode == 0 and run.stdout.startswith("done"), run.stderr[-2000:]


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,heads,dim,rotary,interleaved", [(1, 8, 64, 64, False), (5, 8, 64, 32, False), (700, 4, 128, 128, True),
                                                                 (3, 2, 66, 30, False), (40, 3, 96, 24, True), (2, 5, 80, 80, False)])
@pytest.mark.parametrize("order", ["token", "head"])
def test_fused_projection_in_place(moe, tokens, heads, dim, rotary, interleaved, order):  # noqa: F811
    """Queries, keys and values of a head side by side, token by token and head by head; values and the rest stay as they are."""
    if order == "token":
        fused = torch.randn(tokens, heads, 3, dim, device="cuda").to(torch.bfloat16)
        q, k, v = (fused[:, :, i] for i in range(3))
    else:
        fused = torch.randn(heads, 3, tokens, dim, device="cuda").to(torch.bfloat16)
        q, k, v = (fused[:, i].transpose(0, 1) for i in range(3))
    positions = torch.randint(0, 1 << 20, (tokens,), device="cuda").int()
    turns = moe.moe_rope_turns(rotary, 1e6, device="cuda")
    before = [t.clone() for t in (q, k, v)]
    moe.moe_rope(positions, turns, q, k, interleaved=interleaved)
    for got, x in zip((q, k), before):
        check(got, *rotate(x, positions, turns, interleaved))
        assert torch.equal(got[..., rotary:], x[..., rotary:])
    assert torch.equal(v, before[2])
    # Keys into the values' place, queries where they are.
    moe.moe_rope(positions, turns, q, k, k_out=v, interleaved=interleaved)
    again = torch.empty_like(before[1])
    moe.moe_rope(positions, turns, k, q_out=again, interleaved=interleaved)
    assert torch.equal(v, again)
    for bad in (dict(k=q), dict(k=k, k_out=q), dict(k=k, q_out=k)):
        with pytest.raises(moe.MoeError):
            moe.moe_rope(positions, turns, q, **bad)
