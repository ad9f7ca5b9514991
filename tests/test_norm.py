"""moe_norm against the formula in 64 bits.

Tolerances, derived before their first run (u = 2^-24, FP32's unit roundoff):
a thread sums up to 32 squares one by one, a tree of at most 10 levels joins them
and the quotient and eps add 2 roundings, half of all that in the square root:
22 u; rsqrtf is within 2 ulp (4 u), h one rounding, the products with it and the
weight and the weight's offset 3 more. 40 u relative is above their sum. An output
is rounded once: half a step of its type, relative to it, or of its subnormal
step. A code is half a step of e4m3 (2^-4 relative, 2^-10 under its normal range)
off; its block's scale is the smallest power that holds the block's largest
magnitude, known to 40 u.
"""
from __future__ import annotations

import ctypes

import pytest
import torch

U = 2.0 ** -24
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__

    __graft_entry__.build()
    import mxfp4_weight_mxfp8_gb300 as moe

    return moe


# ------------------------------------------------------------------- refusals
def block(moe, **changes):
    """Arguments of a good call of two rows (nothing is launched with these pointers)."""
    b = moe._Norm(x=0x10000, x_stride=64, weight=0x20000, out=0x30000, out_stride=64, dtype=1, residual_dtype=1,
                  weight_dtype=0, tokens=2, hidden=64, eps=1e-6)
    for k, v in changes.items():
        setattr(b, k, v)
    return b


@pytest.mark.parametrize("changes", [
    dict(tokens=-1), dict(hidden=0), dict(hidden=16385), dict(dtype=3), dict(weight_dtype=-1),
    dict(residual=0x40000, residual_stride=64, residual_dtype=7), dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(weight_offset=float("inf")), dict(codes=0x50000), dict(scales=0x50000), dict(hidden=60, codes=0x50000, scales=0x60000),
    dict(x_stride=-64), dict(residual=0x40000, residual_stride=-1), dict(out_stride=63),
    dict(residual_out=0x40000, residual_out_stride=10), dict(x=0), dict(weight=0), dict(out=0), dict(x=0x10001), dict(out=0x30001),
    dict(weight=0x20002), dict(codes=0x50004, scales=0x60000), dict(out=0x10002), dict(out=0x10000, x_stride=65),
    dict(residual=0x40000, residual_stride=64, residual_out=0x40002, residual_out_stride=64),
    dict(residual=0x40000, residual_stride=64, residual_out=0x10000, residual_out_stride=64),
    dict(residual_out=0x30000, residual_out_stride=64), dict(codes=0x30000, scales=0x60000), dict(codes=0x50000, scales=0x50040),
    dict(out=0x20000)])
def test_norm_refusals(moe, changes):
    with pytest.raises(moe.MoeError) as e:
        moe._check(moe.library().moe_norm(ctypes.byref(block(moe, **changes)), None), "moe_norm")
    assert e.value.code == moe.MOE_ERR_ARG and moe.moe_last_error_detail()


def test_norm_of_no_rows_is_no_work(moe):
    assert moe.library().moe_norm(ctypes.byref(block(moe, tokens=0, x=0, weight=0, out=0)), None) == moe.MOE_OK
    assert moe.library().moe_norm(None, None) == moe.MOE_ERR_ARG


def test_norm_quantize_refuses_without_a_handle(moe):
    assert moe.library().moe_norm_quantize(None, ctypes.byref(block(moe)), None) == moe.MOE_ERR_ARG


def test_packed_blocks_are_as_long_as_the_structs(moe):
    for packed, struct in ((moe._NORM, moe._Norm), (moe._ROPE, moe._Rope), (moe._FORK, moe._KvFork), (moe._RECLAIM, moe._KvReclaim)):
        assert packed.size == ctypes.sizeof(struct)


# -------------------------------------------------------------------- numerics
def reference(x, weight, residual, eps, offset):
    h = x.double()
    if residual is not None:
        h = h + residual.double()
    return h, h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps) * (weight.double() + offset)


def close(got, want, extra=40 * U):
    """Rounded once to its type, from a value within `extra` of the wanted one."""
    info = torch.finfo(got.dtype)
    err = (got.double() - want).abs()
    limit = (info.eps / 2 * (1 + extra) + extra) * want.abs() + info.tiny * info.eps
    fits = want.abs() <= info.max
    bad = fits & ~(err <= limit)
    assert not bad.any(), (err[bad][:4], want[bad][:4])
    return fits


def check_codes(codes, scales, y):
    v = codes.view(torch.float8_e4m3fn).double().view(y.shape[0], -1, 32)
    E = scales.double() - 127
    y = y.view_as(v)
    top = y.abs().amax(-1)
    assert (top * (1 - 40 * U) <= 448 * torch.exp2(E)).all()
    assert ((top * (1 + 40 * U) > 448 * torch.exp2(E - 1)) | (E == -127)).all()
    want = y * torch.exp2(-E)[..., None]
    limit = torch.maximum(want.abs() * 2.0 ** -4, torch.full_like(want, 2.0 ** -10)) * (1 + 64 * U) + 40 * U * want.abs()
    assert ((v - want).abs() <= limit).all()


SHAPES = [(1, 1), (3, 7), (5, 31), (1, 32), (2, 64), (257, 128), (33, 256), (9, 264), (7, 512), (4, 520), (6, 1000), (5, 1024),
          (3, 1032), (64, 3584), (1, 3584), (2, 4099), (3, 8192), (2, 16384), (1, 16383), (1200, 96)]


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hidden", SHAPES)
@pytest.mark.parametrize("dtype,res,wt", [("bfloat16", None, "float32"), ("bfloat16", "bfloat16", "bfloat16"), ("bfloat16", "float32", "float32"),
                                          ("float16", "float16", "float16"), ("float32", None, "float32"), ("float32", "float32", "bfloat16"),
                                          ("float16", "float32", "float32"), ("float32", "bfloat16", "float32")])
def test_norm_matches_64_bits(moe, tokens, hidden, dtype, res, wt):
    g = torch.Generator(device="cuda").manual_seed(tokens * 7 + hidden)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").to(TYPES[dtype])
    w = (1 + 0.3 * torch.randn(hidden, generator=g, device="cuda")).to(TYPES[wt])
    residual = res_out = None
    if res:
        residual = (4 * torch.randn(tokens, hidden, generator=g, device="cuda")).to(TYPES[res])
        res_out = torch.full_like(residual, 7)
    out = torch.full_like(x, 7)
    mx = hidden % 32 == 0
    codes = torch.zeros(tokens, hidden, dtype=torch.uint8, device="cuda") if mx else None
    scales = torch.zeros(tokens, hidden // 32, dtype=torch.uint8, device="cuda") if mx else None
    before = x.clone()
    moe.moe_norm(x, w, out, eps=1e-5, residual=residual, residual_out=res_out, codes=codes, scales=scales, weight_offset=0.25)
    h, y = reference(x, w, residual, 1e-5, 0.25)
    close(out, y)
    if res:
        close(res_out, h, 2 * U)
    if mx:
        check_codes(codes, scales, y)
    assert torch.equal(x, before)


@pytest.mark.gpu
@pytest.mark.parametrize("outputs", ["out", "codes", "both", "out+residual"])
def test_norm_outputs_do_not_depend_on_each_other(moe, outputs):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(19, 2048, generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn(19, 2048, generator=g, device="cuda")
    w = torch.randn(2048, generator=g, device="cuda")

    def call(out, codes, res_out):
        o = torch.zeros_like(x) if out else None
        c = torch.zeros(19, 2048, dtype=torch.uint8, device="cuda") if codes else None
        s = torch.zeros(19, 64, dtype=torch.uint8, device="cuda") if codes else None
        ro = torch.zeros_like(r) if res_out else None
        moe.moe_norm(x, w, o, residual=r, residual_out=ro, codes=c, scales=s)
        return o, c, s, ro

    full = call(True, True, True)
    part = call("out" in outputs or outputs == "both", outputs in ("codes", "both"), "residual" in outputs)
    for a, b in zip(full, part):
        assert b is None or torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("hidden", [64, 3584, 4100])
def test_norm_strides_alignment_and_in_place(moe, hidden):
    g = torch.Generator(device="cuda").manual_seed(hidden)
    wide = torch.randn(11, hidden + 24, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(hidden, generator=g, device="cuda")
    r = torch.randn(11, hidden, generator=g, device="cuda").to(torch.bfloat16)
    plain = torch.empty(11, hidden, dtype=torch.bfloat16, device="cuda")
    for at in (0, 8, 3):  # aligned to 16 bytes and not
        x = wide[:, at:at + hidden]
        moe.moe_norm(x.contiguous(), w, plain, residual=r)
        strided = torch.zeros(11, hidden + 5, dtype=torch.bfloat16, device="cuda")
        moe.moe_norm(x, w, strided[:, 2:hidden + 2], residual=r)
        assert torch.equal(strided[:, 2:hidden + 2], plain)
        assert not strided[:, :2].any() and not strided[:, hidden + 2:].any()
        x2, r2 = wide.clone(), r.clone()
        moe.moe_norm(x2[:, at:at + hidden], w, x2[:, at:at + hidden], residual=r2, residual_out=r2)
        assert torch.equal(x2[:, at:at + hidden], plain)
        assert torch.equal(x2[:, :at], wide[:, :at]) and torch.equal(x2[:, at + hidden:], wide[:, at + hidden:])
        assert torch.equal(r2, (x.float() + r.float()).to(torch.bfloat16))
    # One row for all, read with a stride of 0.
    x = wide[:1, :hidden].expand(11, hidden)
    moe.moe_norm(x, w, plain)
    assert torch.equal(plain, plain[:1].expand(11, hidden))
    # Columns of one buffer, side by side.
    both = torch.zeros(11, 2 * hidden, dtype=torch.bfloat16, device="cuda")
    both[:, :hidden] = wide[:, :hidden]
    moe.moe_norm(both[:, :hidden], w, both[:, hidden:])
    moe.moe_norm(wide[:, :hidden].contiguous(), w, plain)
    assert torch.equal(both[:, hidden:], plain)


@pytest.mark.gpu
@pytest.mark.parametrize("hidden", [96, 3584])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_norm_magnitudes_from_the_smallest_to_the_largest(moe, hidden, dtype):
    rows = torch.tensor([1e-38, 1e-30, 1e-20, 1e-4, 1.0, 1e10, 1e18, 1e19, 1e25, 3e36, 3e38], device="cuda")[:, None]
    g = torch.Generator(device="cuda").manual_seed(2)
    x = (torch.rand(11, hidden, generator=g, device="cuda") * 2 - 1).mul(rows).to(TYPES[dtype])
    w = torch.ones(hidden, device="cuda")
    out = torch.empty_like(x)
    codes = torch.zeros(11, hidden, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(11, hidden // 32, dtype=torch.uint8, device="cuda")
    for eps in (1e-6, 1e-30, 1e30):
        moe.moe_norm(x, w, out, eps=eps, codes=codes, scales=scales)
        y = reference(x, w, None, float(torch.tensor(eps)), 0.0)[1]
        # Squares below FP32's range lose what eps is far above.
        assert close(out, y, 64 * U).all()
        kept = y.abs().view(11, -1, 32).amax((1, 2)) > 1e-30
        check_codes(codes[kept], scales[kept], y[kept])


@pytest.mark.gpu
def test_norm_of_as_many_rows_as_there_can_be(moe):
    """2^31 - 1 rows of one element (4 GB), from an input that is broadcast."""
    x = torch.full((1, 1), 3.0, dtype=torch.bfloat16, device="cuda").expand(2 ** 31 - 1, 1)
    out = torch.zeros(2 ** 31 - 1, 1, dtype=torch.bfloat16, device="cuda")
    moe.moe_norm(x, torch.full((1,), 0.5, device="cuda"), out, 1e-6)  # 3 * 0.5 / sqrt(9 + 1e-6): 0.5 in BF16
    assert (out == 0.5).all()


@pytest.mark.gpu
@pytest.mark.parametrize("hidden", [64, 1000, 3584])
def test_norm_zeros_infinities_and_nan(moe, hidden):
    x = torch.ones(5, hidden, dtype=torch.bfloat16, device="cuda")
    x[0] = 0
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x[3, 7] = float("-inf")
    w = torch.ones(hidden, device="cuda")
    out = torch.empty_like(x)
    moe.moe_norm(x, w, out)
    assert not out[0].any() and torch.isnan(out[2]).all()
    for row, at in ((1, 3), (3, 7)):
        assert torch.isnan(out[row, at])
        rest = torch.cat((out[row, :at], out[row, at + 1:]))
        assert not rest.any()
    assert torch.equal(out[4], torch.ones_like(out[4]))  # a row of ones beside them
    if hidden % 32 == 0:
        codes = torch.zeros(5, hidden, dtype=torch.uint8, device="cuda")
        scales = torch.zeros(5, hidden // 32, dtype=torch.uint8, device="cuda")
        moe.moe_norm(x, w, codes=codes, scales=scales)
        assert not codes[0].any() and not scales[0].any()
        assert ((codes[2] & 127) == 127).all() and (codes[1, 3] & 127) == 127
        assert not (codes[1, :3] & 127).any()


@pytest.mark.gpu
def test_norm_codes_take_the_layers_rule(moe):
    """Codes of rows whose y is exact in BF16 are moe_quantize's of them, bit for bit."""
    import workload

    layer = moe.MoeLayer(tuple(torch.from_numpy(w).cuda() for w in workload.make_weights(16, 256, 32, seed13=1, seed2=2)))
    x = torch.randint(-120, 121, (5, 256), device="cuda").float()
    x = x / x.square().sum(-1, keepdim=True).sqrt()  # any rows: with a weight of 0 and an offset the norm is exact below
    x = torch.where(torch.rand(5, 256, device="cuda") < 0.5, 1.0, -1.0).to(torch.bfloat16)  # mean square 1
    w = torch.exp2(torch.randint(-9, 9, (256,), device="cuda").float()) * (1 + torch.randint(0, 128, (256,), device="cuda") / 128)
    out = torch.empty_like(x)
    codes, scales = (torch.zeros(5, n, dtype=torch.uint8, device="cuda") for n in (256, 8))
    moe.moe_norm(x, w, out, eps=1e-30, codes=codes, scales=scales)
    assert torch.equal(out.float(), x.float() * w)
    import numpy as np

    moe.moe_quantize(layer.handle, out, 5)
    torch.cuda.synchronize()
    want, want_scales = np.empty((5, 256), np.uint8), np.empty((5, 8), np.uint8)
    moe.moe_copy_plan(layer.handle, want, want_scales, 5)
    assert (codes.cpu().numpy() == want).all() and (scales.cpu().numpy() == want_scales).all()
    layer.close()


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [1, 7, 40])
def test_norm_quantize_feeds_the_experts(moe, tokens):
    import numpy as np
    import oracle
    import workload

    weights = workload.make_weights(32, 256, 64, seed13=3, seed2=4)
    layer = moe.MoeLayer(tuple(torch.from_numpy(w).cuda() for w in weights))
    ids = workload.make_ids(tokens, 32, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(tokens, 256, generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn(tokens, 256, generator=g, device="cuda").to(torch.bfloat16)
    w = 1 + 0.1 * torch.randn(256, generator=g, device="cuda")
    normed, res, rows = torch.empty_like(x), torch.empty_like(r), torch.empty(tokens, 16, 256, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        moe.moe_norm_quantize(layer.handle, x, w, normed, residual=r, residual_out=res)
        moe.moe_group(layer.handle, torch.from_numpy(ids).cuda(), tokens)
        moe.moe_experts(layer.handle, rows, tokens)
    assert moe.moe_sync_status(layer.handle) == moe.MOE_OK
    codes, scales = np.empty((tokens, 256), np.uint8), np.empty((tokens, 8), np.uint8)
    moe.moe_copy_plan(layer.handle, codes, scales, tokens)
    y = reference(x, w, r, 1e-6, 0.0)[1]
    check_codes(torch.from_numpy(codes), torch.from_numpy(scales), y.cpu())
    close(normed, y)
    want = oracle.pairs_forward(weights, codes, scales, ids)["out"]
    want = torch.from_numpy(want.view(np.int16)).view(torch.bfloat16).double()
    got = rows.cpu().double().view(tokens * 16, 256)
    assert torch.linalg.norm(got - want) <= 1e-2 * torch.linalg.norm(want)
    for bad in (dict(x=x[:, :128], weight=w[:128]), dict(x=x.repeat(300, 1)[:257], weight=w)):
        with pytest.raises(moe.MoeError):
            moe.moe_norm_quantize(layer.handle, bad["x"], bad["weight"])
    layer.close()


@pytest.mark.gpu
def test_norm_on_a_stream_in_a_graph_and_row_independence(moe):
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(300, 3584, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(3584, generator=g, device="cuda")
    out, one = torch.empty_like(x), torch.empty_like(x[:1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_norm(x, w, out, stream=side)
    side.synchronize()
    for t in (0, 131, 299):
        moe.moe_norm(x[t:t + 1], w, one)
        assert torch.equal(one[0], out[t])
    graph = torch.cuda.CUDAGraph()
    again = torch.empty_like(x)
    with torch.cuda.graph(graph):
        moe.moe_norm(x, w, again)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out)
    x.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, -out)


@pytest.mark.gpu
def test_norm_python_refusals(moe):
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    for bad in (lambda: moe.moe_norm(x.cpu(), w, x), lambda: moe.moe_norm(x, w.cpu(), x), lambda: moe.moe_norm(x, w, x.float()),
                lambda: moe.moe_norm(x.t(), w, x), lambda: moe.moe_norm(x, w[:32], x), lambda: moe.moe_norm(x.int(), w, x),
                lambda: moe.moe_norm(x, w, x, residual=x.float(), residual_out=x.clone()), lambda: moe.moe_norm(x, w),
                lambda: moe.moe_norm(x, w, codes=torch.zeros(2, 64, dtype=torch.uint8, device="cuda")),
                lambda: moe.moe_norm(x[0], w, x[0])):
        with pytest.raises(moe.MoeError) as e:
            bad()
        assert e.value.code == moe.MOE_ERR_ARG
