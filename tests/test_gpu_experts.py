"""GPU parity of the expert layer behind the router against fp64: grouping of the pairs,
grouped products in bf16 and MXFP4 with and without SwiGLU, the weighted combine, and a
whole layer from the router to the combined output."""
import numpy as np
import pytest
import torch

from experts_common import (bf16_normal, check, linear_bound, mxfp4_normal, sizes_to_offsets,
                            swiglu_bound)
from gpu_common import dev, host, require_gpu
from oracle import experts

pytestmark = pytest.mark.gpu

SA_OK, SA_ERR_BOUNDS, SA_ERR_TIMEOUT = 0, 5, 6
ALPHA, LIMIT = 1.702, 7.0


# ----------------------------------------------------------------------------- grouping
@pytest.mark.parametrize("t,k,e", [(0, 4, 128), (1, 1, 1), (1, 4, 128), (7, 8, 8), (33, 2, 31), (64, 4, 128),
                                   (1024, 4, 256), (1025, 4, 32), (4097, 3, 100), (32768, 4, 128), (20001, 8, 255)])
@pytest.mark.parametrize("padded", [False, True])
def test_group_rows(t, k, e, padded):
    sa = require_gpu()
    rng = np.random.default_rng(1000 * t + 10 * k + e)
    idx = rng.integers(0, e, (t, k)).astype(np.int32)  # a token may name an expert twice
    if padded:  # padded tokens, and single pairs without expert
        idx[rng.random(t) < 0.3] = -1
        idx[rng.random((t, k)) < 0.1] = -7
    ref = experts.group_rows(idx, e)
    got = sa.moe_group_rows(dev(idx), e)
    for g, r, name in zip(got, ref, ("expert_offsets", "row_token", "pair_row")):
        assert np.array_equal(g.cpu().numpy(), r), name
    assert sa.sink_attn_device_status(True) == SA_OK


def test_group_rows_one_expert_takes_all_and_large_indices_are_reported():
    sa = require_gpu()
    sa.sink_attn_device_status(True)
    idx = np.full((5000, 4), 17, dtype=np.int32)
    off, tok, row = sa.moe_group_rows(dev(idx), 64)
    assert np.array_equal(off.cpu().numpy(), np.where(np.arange(65) > 17, 20000, 0))
    assert np.array_equal(row.cpu().numpy().reshape(-1), np.arange(20000))
    assert np.array_equal(tok.cpu().numpy(), np.arange(20000) // 4)
    assert sa.sink_attn_device_status(True) == SA_OK
    idx[3, 2], idx[4999, 0] = 64, 2 ** 31 - 1
    ref = experts.group_rows(idx, 64)
    got = sa.moe_group_rows(dev(idx), 64)
    assert all(np.array_equal(g.cpu().numpy(), r) for g, r in zip(got, ref))
    assert sa.sink_attn_device_status(True) == SA_ERR_BOUNDS


# ----------------------------------------------------------------------------- products
def _operands(rng, mx, rows, e, n, k, std=None):
    """((call's operands), x, w) with x [rows, k] and w [e, n, k]."""
    std = 1.0 / np.sqrt(k) if std is None else std
    if mx:
        xc, xs, xv = mxfp4_normal(rng, (rows, k))
        wc, ws, wv = mxfp4_normal(rng, (e, n, k), std)
        return (xc, xs, wc, ws), xv, wv
    x, xv = bf16_normal(rng, (rows, k))
    w, wv = bf16_normal(rng, (e, n, k), std)
    return (x, w), xv, wv


def _call(sa, mx, act, operands, offsets, **kw):
    name = ("grouped_mxfp4_linear_" if mx else "grouped_linear_") + ("swiglu" if act else "bias")
    return getattr(sa, name)(*operands, offsets, **kw)


def _reference(xv, wv, bv, offsets, row_token, act, k, alpha=ALPHA, limit=LIMIT):
    y, mag = experts.grouped_linear(xv, wv, bv, offsets, row_token)
    if act:
        return experts.swiglu(y, alpha, limit), swiglu_bound(y, mag, k, alpha, limit)
    return y, linear_bound(y, mag, k)


CASES = [  # experts' row counts, features, inputs (bf16, MXFP4)
    ([1], 2, (8, 32)),
    ([0, 1, 17, 0], 130, (72, 96)),
    ([128, 129, 0, 113, 257, 1], 300, (200, 544)),
    ([112, 224, 225, 15, 16], 514, (264, 256)),
    ([1, 0, 0, 2, 1, 0, 0, 0], 2880, (2880, 2880)),
    ([700, 5, 1300], 642, (1048, 1056)),
    (list(np.random.default_rng(3).integers(0, 4, 256)), 128, (64, 64)),
    ([2300, 3, 4700], 300, (72, 96)),           # more than eight row tiles: several bands of them
    ([49, 51, 33, 64, 65, 40], 1000, (136, 320)),   # about 48 rows per expert: single CTAs, 1 and 2 row tiles
]


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp4"])
@pytest.mark.parametrize("act", [False, True], ids=["bias", "swiglu"])
@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gather"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_grouped_products(case, gather, act, mx):
    sa = require_gpu()
    sa.sink_attn_device_status(True)
    sizes, n, k = CASES[case]
    k = k[1] if mx else k[0]
    rng = np.random.default_rng(100 + case)
    e, start, behind = len(sizes), 3, 5
    offsets = sizes_to_offsets(sizes, start)  # rows before the first group and behind the last
    rows = int(offsets[-1]) + behind
    x_rows = 41 if gather else rows
    row_token = rng.integers(0, x_rows, rows).astype(np.int32) if gather else None
    operands, xv, wv = _operands(rng, mx, x_rows, e, n, k)
    bias, bv = bf16_normal(rng, (e, n)) if case % 2 else (None, None)
    outside = torch.full((rows, n // 2 if act else n), 7.5, dtype=torch.bfloat16, device="cuda")
    out = _call(sa, mx, act, operands, dev(offsets), bias=bias, out=outside.clone(),
                row_token=None if row_token is None else dev(row_token))
    ref, bound = _reference(xv, wv, bv, offsets, row_token, act, k)
    check(host(out), ref, bound, f"case {case} gather={gather} act={act} mxfp4={mx}")
    keep = torch.ones(rows, dtype=torch.bool)
    keep[start:rows - behind] = False
    assert torch.equal(out[keep.cuda()], outside[keep.cuda()]), "rows outside the groups were written"
    assert sa.sink_attn_device_status(True) == SA_OK


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp4"])
def test_grouped_many_tiles_per_cta(mx):
    """Far more tiles than SMs, so every CTA goes round its ring and both accumulators many
    times; the reference is an fp64 product on the GPU, expert by expert."""
    sa = require_gpu()
    rng = np.random.default_rng(5)
    e, n, k, t = 24, 2880, 1440, 3001
    idx = dev(np.argsort(rng.random((t, e)) + 0.2 * rng.standard_normal(e), axis=1)[:, :4].astype(np.int32))
    offsets, row_token, _ = sa.moe_group_rows(idx, e)
    operands, xv, wv = _operands(rng, mx, t, e, n, k)
    bias, bv = bf16_normal(rng, (e, n))
    x, w, b = (torch.from_numpy(v).cuda() for v in (xv, wv, bv))
    ends = offsets.tolist()
    for act in (False, True):
        out = _call(sa, mx, act, operands, offsets, bias=bias, row_token=row_token)
        for i in range(e):
            at = row_token[ends[i]:ends[i + 1]].long()
            y = (x[at] @ w[i].T + b[i]).cpu().numpy()
            mag = (x[at].abs() @ w[i].abs().T + b[i].abs()).cpu().numpy()
            ref, bound = (experts.swiglu(y, ALPHA, LIMIT), swiglu_bound(y, mag, k, ALPHA, LIMIT)) if act else \
                (y, linear_bound(y, mag, k))
            check(host(out[ends[i]:ends[i + 1]]), ref, bound, f"expert {i} act={act} mxfp4={mx}")
    assert sa.sink_attn_device_status(True) == SA_OK


@pytest.mark.parametrize("m,n,k", [(0, 64, 64), (1, 1, 32), (1, 2880, 2880), (112, 128, 256), (113, 257, 288),
                                   (1000, 640, 4096), (640, 5120, 96)])
def test_mxfp4_linear(m, n, k):
    sa = require_gpu()
    rng = np.random.default_rng(m + n + k)
    xc, xs, xv = mxfp4_normal(rng, (m, k))
    wc, ws, wv = mxfp4_normal(rng, (n, k), 1.0 / np.sqrt(k))
    bias, bv = bf16_normal(rng, (n,))
    for b, v in ((bias, bv), (None, None)):
        out = sa.mxfp4_linear_bias(xc, xs, wc, ws, b)
        assert out.shape == (m, n)
        if m:
            ref, mag = experts.grouped_linear(xv, wv[None], None if v is None else v[None], [0, m])
            check(host(out), ref, linear_bound(ref, mag, k), f"mxfp4 {m}x{n}x{k}")
    assert sa.sink_attn_device_status(True) == SA_OK


def test_mxfp4_scales_of_every_size_and_nan():
    """Blocks whose scales differ by up to 2^60 within a row, and a NaN scale: exactly the
    products with that block are NaN."""
    sa = require_gpu()
    rng = np.random.default_rng(9)
    m, n, k = 150, 200, 640
    xc, xs, _ = mxfp4_normal(rng, (m, k))
    wc, ws, _ = mxfp4_normal(rng, (n, k))
    xs[:, : k // 32] = torch.from_numpy(rng.integers(97, 157, (m, k // 32)).astype(np.uint8))
    ws[:, : k // 32] = torch.from_numpy(rng.integers(97, 157, (n, k // 32)).astype(np.uint8))
    val = lambda c, s: experts.mxfp4_dequantize(c.cpu().numpy(), s.cpu().numpy())  # noqa: E731
    ref, mag = experts.grouped_linear(val(xc, xs), val(wc, ws)[None], None, [0, m])
    out = sa.mxfp4_linear_bias(xc, xs, wc, ws)
    assert np.all(np.abs(host(out) - ref) <= linear_bound(ref, mag, k))
    xs[7, 3], ws[130, 19] = 255, 255
    out = host(sa.mxfp4_linear_bias(xc, xs, wc, ws))
    nan = np.zeros((m, n), dtype=bool)
    nan[7], nan[:, 130] = True, True
    assert np.array_equal(np.isnan(out), nan)


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp4"])
def test_rows_do_not_touch_one_another(mx):
    """NaN in rows of x that no group reads, or that other rows read, stays where it is."""
    sa = require_gpu()
    rng = np.random.default_rng(11)
    e, n, k, x_rows = 3, 256, 512, 50
    sizes = [20, 0, 33]
    offsets = sizes_to_offsets(sizes, 2)
    rows = int(offsets[-1]) + 4
    row_token = rng.integers(1, x_rows, rows).astype(np.int32)
    row_token[[2, 30]] = 0           # two rows read the NaN row
    row_token[:2], row_token[-4:] = -5, 10 ** 9   # outside the groups: never read
    operands, _, _ = _operands(rng, mx, x_rows, e, n, k)
    (operands[1] if mx else operands[0])[0] = 255 if mx else float("nan")
    for act in (False, True):
        out = _call(sa, mx, act, operands, dev(offsets), row_token=dev(row_token))
        bad = torch.isnan(out[2:-4]).all(1).cpu().numpy()
        assert np.array_equal(np.nonzero(bad)[0], [0, 28])
        assert not torch.isnan(out[2:-4][torch.from_numpy(~bad).cuda()]).any()
    assert sa.sink_attn_device_status(True) == SA_OK


def test_swiglu_clamps_limits_and_infinities():
    """The activation at, beyond and far beyond its clamps, and without a clamp: gate and up
    values are given exactly through the bias (x = 0)."""
    sa = require_gpu()
    g = np.array([-1e30, -300.0, -88.0, -20.0, -7.0, -1.0, -0.0, 0.0, 1e-20, 0.5, 6.96875, 7.0, 7.03125, 50.0, 1e30])
    u = np.array([-1e30, -7.03125, -7.0, -1.0, 0.0, 3.0, 7.0, 1e30])
    gg, uu = (v.reshape(-1) for v in np.meshgrid(g, u))
    y = np.stack([gg, uu], -1).reshape(1, -1)
    bias = torch.from_numpy(y).to(torch.bfloat16).cuda()
    y = bias.double().cpu().numpy()
    x = torch.zeros((1, 8), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((1, y.shape[1], 8), dtype=torch.bfloat16, device="cuda")
    off = dev(np.array([0, 1], dtype=np.int32))
    for alpha, limit in ((1.702, 7.0), (1.0, 0.5), (1.702, float("inf")), (0.0, 7.0), (-2.0, 3.0)):
        with np.errstate(over="ignore", invalid="ignore"):
            ref = experts.swiglu(y, alpha, limit)
            bound = swiglu_bound(y, np.abs(y), 8, alpha, limit)
        got = host(sa.grouped_linear_swiglu(x, w, off, bias, alpha=alpha, limit=limit))
        fine = np.isfinite(ref) & (np.abs(ref) < 3e38)
        assert np.all(np.abs(got[fine] - ref[fine]) <= bound[fine]), (alpha, limit)
    nan = torch.full_like(bias, float("nan"))
    assert torch.isnan(sa.grouped_linear_swiglu(x, w, off, nan)).all()


@pytest.mark.parametrize("n", [16, 18], ids=["wide", "narrow"])
def test_swiglu_of_huge_alpha(n):
    """Any finite alpha: sigmoid becomes a step, and a gate of 0 still gives 0 (0 times an
    overflowed alpha would be NaN).  With x = 0 the products are the bias: whole numbers, exact."""
    sa = require_gpu()
    x = torch.zeros((3, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((1, n, 64), dtype=torch.bfloat16, device="cuda")
    gate = np.resize([0.0, 1.0, -1.0, 2.0], n // 2)
    bias = torch.from_numpy(np.stack([gate, np.ones(n // 2)], 1).reshape(1, n)).to(torch.bfloat16).cuda()
    for alpha in (3e38, -3e38, 0.0):
        out = host(sa.grouped_linear_swiglu(x, w, dev(np.array([0, 3], dtype=np.int32)), bias, alpha=alpha))
        sigmoid = np.where(gate * alpha > 0, 1.0, np.where(gate * alpha < 0, 0.0, 0.5))
        assert np.array_equal(out, np.broadcast_to(gate * sigmoid * 2.0, out.shape))


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp4"])
def test_bad_groups_and_bad_rows_are_reported_and_skipped(mx):
    sa = require_gpu()
    sa.sink_attn_device_status(True)
    rng = np.random.default_rng(13)
    e, n, k, rows = 4, 200, 256, 60
    operands, xv, wv = _operands(rng, mx, rows, e, n, k)
    good = np.array([0, 20, 20, 45, 60], dtype=np.int32)
    ref, bound = _reference(xv, wv, None, good, None, False, k)
    # offsets, and the groups that still count
    for offsets, kept in (([0, 20, 20, 45, 61], [0, 2]), ([-1, 20, 20, 45, 60], [2, 3]),
                          ([0, 20, 10, 45, 60], [0, 3]), ([0, 2 ** 30, 20, 45, 60], [])):
        filled = torch.full((rows, n), 3.0, dtype=torch.bfloat16, device="cuda")
        out = host(_call(sa, mx, False, operands, dev(np.array(offsets, dtype=np.int32)), out=filled))
        assert sa.sink_attn_device_status(True) == SA_ERR_BOUNDS, offsets
        for i in range(e):
            at = slice(int(good[i]), int(good[i + 1]))
            if i in kept:
                assert np.all(np.abs(out[at] - ref[at]) <= bound[at]), (offsets, i)
            else:
                assert np.all(out[at] == 3.0), (offsets, i)
    # a row index outside x: reported, every other row right
    row_token = rng.permutation(rows).astype(np.int32)
    ref, bound = _reference(xv, wv, None, good, row_token, False, k)
    bad = row_token.copy()
    bad[33], bad[2] = rows, -1
    out = host(_call(sa, mx, False, operands, dev(good), row_token=dev(bad)))
    assert sa.sink_attn_device_status(True) == SA_ERR_BOUNDS
    others = np.setdiff1d(np.arange(rows), [2, 33])
    assert np.all(np.abs(out[others] - ref[others]) <= bound[others])


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp4"])
def test_zero_wait_budget_unwinds_cleanly(mx):
    sa = require_gpu()
    sa.sink_attn_device_status(True)
    rng = np.random.default_rng(15)
    sizes = [300, 40, 500, 1]
    offsets = sizes_to_offsets(sizes)
    operands, xv, wv = _operands(rng, mx, int(offsets[-1]), 4, 640, 1024)
    try:
        sa.sink_attn_set_wait_timeout_ns(0)
        _call(sa, mx, False, operands, dev(offsets))
        assert sa.sink_attn_device_status(True) in (SA_OK, SA_ERR_TIMEOUT)
    finally:
        sa.sink_attn_set_wait_timeout_ns(2_000_000_000)
    out = _call(sa, mx, False, operands, dev(offsets))
    ref, bound = _reference(xv, wv, None, offsets, None, False, 1024)
    check(host(out), ref, bound, "after a zero wait budget")
    assert sa.sink_attn_device_status(True) == SA_OK


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp4"])
@pytest.mark.parametrize("sizes", [[3, 0, 1, 2], [100, 40, 60, 31], [20, 11, 0, 7]], ids=["cap16", "pair", "cap64"])
def test_zero_wait_budget_with_gathered_rows(sizes, mx):
    """As above where threads bring the rows, for each kind of tile."""
    sa = require_gpu()
    sa.sink_attn_device_status(True)
    rng = np.random.default_rng(16)
    offsets = sizes_to_offsets(sizes)
    operands, xv, wv = _operands(rng, mx, 50, 4, 640, 2080)
    token = rng.integers(0, 50, int(offsets[-1])).astype(np.int32)
    try:
        sa.sink_attn_set_wait_timeout_ns(0)
        for _ in range(3):
            _call(sa, mx, False, operands, dev(offsets), row_token=dev(token))
        assert sa.sink_attn_device_status(True) in (SA_OK, SA_ERR_TIMEOUT)
    finally:
        sa.sink_attn_set_wait_timeout_ns(2_000_000_000)
    out = _call(sa, mx, False, operands, dev(offsets), row_token=dev(token))
    ref, bound = _reference(xv, wv, None, offsets, token, False, 2080)
    check(host(out), ref, bound, "after a zero wait budget")
    assert sa.sink_attn_device_status(True) == SA_OK


def test_output_at_an_odd_address_and_no_rows():
    """out needs 2-byte alignment only; no rows at all launch nothing."""
    sa = require_gpu()
    rng = np.random.default_rng(17)
    operands, xv, wv = _operands(rng, False, 40, 2, 96, 64)
    offsets = sizes_to_offsets([25, 15])
    buf = torch.zeros(40 * 96 + 1, dtype=torch.bfloat16, device="cuda")
    out = sa.grouped_linear_bias(*operands, dev(offsets), out=buf[1:].view(40, 96))
    ref, bound = _reference(xv, wv, None, offsets, None, False, 64)
    check(host(out), ref, bound, "odd address")
    assert buf[0].item() == 0
    empty = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert sa.grouped_linear_bias(empty, operands[1], dev(np.zeros(3, np.int32))).shape == (0, 96)
    token = torch.empty((0,), dtype=torch.int32, device="cuda")
    assert sa.grouped_linear_swiglu(operands[0], operands[1], dev(np.zeros(3, np.int32)), row_token=token).shape == (0, 48)


def test_beyond_32_bit_offsets():
    """Outputs, weights and gathered sums whose element offsets pass 2^31: the last rows and the
    last experts, against fp64."""
    sa = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(3)
    rows, n, k = 800_000, 2816, 64                        # out: 2.25e9 elements
    x = torch.randn(rows, k, generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(2, n, k, generator=g, device="cuda", dtype=torch.bfloat16) / 8
    off = torch.tensor([0, 300_000, rows], dtype=torch.int32, device="cuda")
    last = slice(rows - 300, rows)
    y = x[last].double().cpu().numpy() @ w[1].double().cpu().numpy().T
    mag = x[last].abs().double().cpu().numpy() @ w[1].abs().double().cpu().numpy().T
    out = sa.grouped_linear_bias(x, w, off)
    check(host(out[last]), y, linear_bound(y, mag, k), "last rows")
    pair_row = torch.tensor([[rows - 1, 5], [rows - 2, rows - 3]], dtype=torch.int32, device="cuda")
    one = torch.ones((2, 2), dtype=torch.bfloat16, device="cuda")
    sums = out[pair_row.long()].double().sum(1)
    # two exact products, one fp32 sum, one rounding to bf16
    assert ((sa.moe_combine(out, pair_row, one).double() - sums).abs() <= (2.0 ** -8 + 2.0 ** -22) * out[
        pair_row.long()].double().abs().sum(1)).all()
    codes, scales = sa.mxfp4_quantize(out)
    tail = [v[last].cpu().numpy() for v in (codes, scales)]
    ref = experts.mxfp4_quantize(host(out[last]))
    assert np.array_equal(tail[0], ref[0]) and np.array_equal(tail[1], ref[1])
    value = experts.mxfp4_dequantize(*ref)
    assert np.array_equal(host(sa.mxfp4_dequantize(codes, scales)[last]), value)
    del out, codes, scales
    e, n, k = 256, 4096, 2112                             # w: 2.2e9 elements
    w = torch.empty(e, n, k, device="cuda", dtype=torch.bfloat16).normal_(std=k ** -0.5, generator=g)
    x = torch.randn(5, k, generator=g, device="cuda", dtype=torch.bfloat16)
    sizes = np.zeros(e, dtype=int)
    sizes[[7, 254, 255]] = 1, 2, 2
    off = sizes_to_offsets(sizes)
    xv = x.double().cpu().numpy()
    for mx in (False, True):
        operands = (*sa.mxfp4_quantize(x), *sa.mxfp4_quantize(w)) if mx else (x, w)
        out = _call(sa, mx, False, operands, dev(off))
        for i in (7, 254, 255):
            at = slice(int(off[i]), int(off[i + 1]))
            xi, wi = xv[at], w[i].double().cpu().numpy()
            if mx:
                xi, wi = (experts.mxfp4_dequantize(*experts.mxfp4_quantize(v)) for v in (xi, wi))
            y, mag = xi @ wi.T, np.abs(xi) @ np.abs(wi).T
            check(host(out[at]), y, linear_bound(y, mag, k), f"expert {i} mxfp4={mx}")
    assert sa.sink_attn_device_status(True) == SA_OK


def test_shapes_and_layouts_are_checked():
    sa = require_gpu()
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    new = lambda *shape, dt=bf: torch.zeros(*shape, dtype=dt, device="cuda")  # noqa: E731
    x, w, off = new(6, 64), new(3, 32, 64), new(4, dt=i32)
    xc, xs, wc, ws = new(6, 32, dt=u8), new(6, 16, dt=u8), new(3, 32, 32, dt=u8), new(3, 32, 16, dt=u8)
    wrong = [
        lambda: sa.grouped_linear_bias(x[:, :56].contiguous(), w, off), lambda: sa.grouped_linear_bias(x[:, :56], w, off),
        lambda: sa.grouped_linear_bias(x, w, off[:3]), lambda: sa.grouped_linear_bias(x, w, off, new(3, 31)),
        lambda: sa.grouped_linear_bias(x, w, off, row_token=new(2, 3, dt=i32)),
        lambda: sa.grouped_linear_bias(x, w, off, out=new(6, 33)), lambda: sa.grouped_linear_swiglu(x, w, off, out=new(6, 32)),
        lambda: sa.grouped_linear_bias(x.t(), w, off), lambda: sa.grouped_linear_bias(x.view(-1), w, off),
        lambda: sa.grouped_mxfp4_linear_bias(xc, xs[:, :2].contiguous(), wc, ws, off),
        lambda: sa.grouped_mxfp4_linear_bias(xc, xs, wc, ws[:2], off), lambda: sa.mxfp4_linear_bias(xc, xs, wc[0], ws[1, :30]),
        lambda: sa.mxfp4_linear_bias(xc, xs, wc[0], ws[0], new(31)), lambda: sa.mxfp4_dequantize(xc, xs[:5]),
        lambda: sa.moe_combine(x, new(2, 3, dt=i32), new(2, 2)), lambda: sa.moe_combine(x, new(2, 3, dt=i32), new(2, 3), out=new(2, 63)),
        lambda: sa.moe_group_rows(new(5, dt=i32), 4), lambda: sa.moe_group_rows(new(5, 2, dt=i32), 4, expert_offsets=new(4, dt=i32)),
        lambda: sa.mxfp4_quantize(x, codes=new(6, 31, dt=u8)),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises(ValueError):
            call()
            print("accepted:", i)
    for call in (lambda: sa.grouped_linear_bias(x.float(), w, off), lambda: sa.moe_group_rows(new(5, 2, dt=torch.int64), 4),
                 lambda: sa.grouped_linear_bias(x, w, off, new(3, 32, dt=torch.float32))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: sa.moe_group_rows(new(5, 9, dt=i32), 4), lambda: sa.mxfp4_quantize(new(4, 40)),
                 lambda: sa.moe_combine(new(6, 60), new(2, 3, dt=i32), new(2, 3)),
                 lambda: sa.grouped_linear_swiglu(x, new(3, 31, 64), off), lambda: sa.grouped_linear_swiglu(x, w, off, limit=0.0)):
        with pytest.raises(sa.SinkAttnError):
            call()
    assert sa.sink_attn_device_status(True) == SA_OK


def test_sizes_past_the_c_interface_are_refused():
    """Sizes that a C int cannot hold raise instead of arriving as what is left of them (2^32 + 64
    values per row would be 64)."""
    sa = require_gpu()
    far = 2 ** 32 + 64
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((2, 32, 64), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    idx = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    long8 = torch.empty(far, dtype=torch.uint8, device="cuda")
    long16 = torch.empty(far, dtype=torch.bfloat16, device="cuda")
    long32 = torch.empty(far, dtype=torch.int32, device="cuda")
    out = torch.empty(1, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: sa.moe_group_rows(idx, 2 ** 32 + 8), lambda: sa.moe_group_rows(idx, 2 ** 31),
                 lambda: sa.grouped_linear_bias(x, w, off, row_token=long32, out=out),
                 lambda: sa.moe_combine(x, long32.view(-1, 1), long16.view(-1, 1), out=out),
                 lambda: sa.mxfp4_quantize(long16.view(1, -1)), lambda: sa.mxfp4_dequantize(long8.view(1, -1), long8)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(sa.SinkAttnError):
        sa.moe_group_rows(idx, -5)
    assert sa.sink_attn_device_status(True) == SA_OK


# ----------------------------------------------------------------------------- combine
@pytest.mark.parametrize("t,k,h", [(1, 1, 8), (1, 4, 2880), (7, 8, 24), (64, 4, 2880), (333, 3, 1000), (3001, 2, 512),
                                   (50, 5, 72), (51, 6, 80), (52, 7, 88)])
def test_combine(t, k, h):
    """fp32 sums of k products (each rounded, at most k + 1 roundings of partial sums bounded by
    sum |w y|), then one bf16 rounding."""
    sa = require_gpu()
    rng = np.random.default_rng(t + k + h)
    rows = t * k + 3
    y, yv = bf16_normal(rng, (rows, h))
    w, wv = bf16_normal(rng, (t, k))
    pair_row = rng.permutation(rows)[: t * k].reshape(t, k).astype(np.int32)
    pair_row[rng.random((t, k)) < 0.2] = -1
    pair_row[0] = -1 if t > 1 else pair_row[0]
    unread = np.setdiff1d(np.arange(rows), pair_row)
    y[torch.from_numpy(unread).cuda()] = float("nan")  # rows without a pair may hold anything
    out = host(sa.moe_combine(y, dev(pair_row), w))
    ref = experts.combine(yv, pair_row, wv)
    mag = experts.combine(np.abs(yv), pair_row, np.abs(wv))
    acc = (k + 1) * 2.0 ** -23 * mag
    assert np.all(np.abs(out - ref) <= acc + 2.0 ** -8 * (np.abs(ref) + acc))
    assert t == 1 or np.all(out[0] == 0)
    assert sa.sink_attn_device_status(True) == SA_OK


def test_combine_rows_out_of_range_are_reported():
    sa = require_gpu()
    sa.sink_attn_device_status(True)
    y = torch.ones((4, 16), dtype=torch.bfloat16, device="cuda")
    w = torch.full((2, 2), 0.5, dtype=torch.bfloat16, device="cuda")
    out = sa.moe_combine(y, dev(np.array([[0, 4], [-2, 3]], dtype=np.int32)), w)
    assert (out == 0.5).all()
    assert sa.sink_attn_device_status(True) == SA_ERR_BOUNDS
    none = sa.moe_combine(y[:0], dev(np.full((3, 2), -1, dtype=np.int32)), w[:1].repeat(3, 1))
    assert (none == 0).all()
    assert sa.sink_attn_device_status(True) == SA_OK


# ----------------------------------------------------------------------------- streams
def _stream_of(t):
    """The stream whose memory pool a tensor's storage belongs to."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in any segment")


def test_outputs_belong_to_the_stream_that_writes_them():
    """With ``stream=`` an output's memory comes from that stream's pool: memory of the current
    stream's pool may still be in use by what runs there, and may be given out there again while
    the kernel writes."""
    sa = require_gpu()
    s = torch.cuda.Stream()
    d = _layer_inputs(sa, 3, 20, 512, 384, 16, 4)
    codes, scales = sa.mxfp4_quantize(d["x"])
    idx, weight = sa.moe_router(d["x"], d["wr"], d["br"], 4)
    offsets, row_token, pair_row = sa.moe_group_rows(idx, 16)
    y = torch.zeros((80, 512), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    outs = [*sa.moe_group_rows(idx, 16, stream=s), sa.moe_combine(y, pair_row, weight, stream=s),
            sa.grouped_linear_swiglu(d["x"], d["up"], offsets, row_token=row_token, stream=s),
            sa.grouped_mxfp4_linear_swiglu(codes, scales, *d["up4"], offsets, row_token=row_token, stream=s),
            sa.mxfp4_linear_bias(codes, scales, d["up4"][0][0], d["up4"][1][0], stream=s),
            *sa.mxfp4_quantize(d["x"], stream=s), sa.mxfp4_dequantize(codes, scales, stream=s)]
    assert [_stream_of(t) for t in outs] == [s.cuda_stream] * len(outs)
    with torch.cuda.stream(s):
        assert _stream_of(sa.mxfp4_dequantize(codes, scales)) == s.cuda_stream
    torch.cuda.synchronize()
    assert sa.sink_attn_device_status(True) == SA_OK


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp4"])
def test_two_graphs_in_turn_and_at_once(mx):
    """Two captured layers of different sizes, replayed in turn and on two streams at once: nothing
    is shared between them."""
    sa = require_gpu()
    d = [_layer_inputs(sa, 60 + t, t, 512, 384, 16, 4) for t in (9, 400)]
    want = [_layer(sa, v, mx)[-1].clone() for v in d]
    graphs, outs = [], []
    for v in d:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_layer(sa, v, mx)[-1])
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for at_once in (False, True) * 3:
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
            if not at_once:
                s.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert sa.sink_attn_device_status(True) == SA_OK


# ----------------------------------------------------------------------------- together
def _layer(sa, d, mx, stream=None):
    """Router to combined output; every intermediate is returned."""
    idx, weight = sa.moe_router(d["x"], d["wr"], d["br"], d["k"], stream=stream)
    offsets, row_token, pair_row = sa.moe_group_rows(idx, d["wr"].shape[0], stream=stream)
    if mx:
        h = sa.grouped_mxfp4_linear_swiglu(*sa.mxfp4_quantize(d["x"], stream=stream), *d["up4"], offsets, d["bu"],
                                           row_token=row_token, stream=stream)
        y = sa.grouped_mxfp4_linear_bias(*sa.mxfp4_quantize(h, stream=stream), *d["down4"], offsets, d["bd"],
                                         stream=stream)
    else:
        h = sa.grouped_linear_swiglu(d["x"], d["up"], offsets, d["bu"], row_token=row_token, stream=stream)
        y = sa.grouped_linear_bias(h, d["down"], offsets, d["bd"], stream=stream)
    return idx, weight, offsets, row_token, pair_row, h, y, sa.moe_combine(y, pair_row, weight, stream=stream)


def _layer_inputs(sa, seed, t, hidden, inner, e, k):
    rng = np.random.default_rng(seed)
    d = {"k": k}
    for name, shape, std in (("x", (t, hidden), 1.0), ("wr", (e, hidden), 0.05), ("br", (e,), 0.5),
                             ("up", (e, 2 * inner, hidden), hidden ** -0.5), ("bu", (e, 2 * inner), 0.5),
                             ("down", (e, hidden, inner), inner ** -0.5), ("bd", (e, hidden), 0.5)):
        d[name], d[name + "_v"] = bf16_normal(rng, shape, std)
    d["up4"], d["down4"] = sa.mxfp4_quantize(d["up"]), sa.mxfp4_quantize(d["down"])
    return d


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp4"])
@pytest.mark.parametrize("t", [1, 37, 600])
def test_layer_from_router_to_combine(t, mx):
    """Each step against fp64 on the step's own inputs, so the bounds are those of one step."""
    sa = require_gpu()
    sa.sink_attn_device_status(True)
    hidden, inner, e, k = 512, 384, 16, 4
    d = _layer_inputs(sa, 21 + t, t, hidden, inner, e, k)
    idx, weight, offsets, row_token, pair_row, h, y, out = _layer(sa, d, mx)
    ref = experts.group_rows(idx.cpu().numpy(), e)
    assert all(np.array_equal(g.cpu().numpy(), r) for g, r in zip((offsets, row_token, pair_row), ref))
    off, tok = ref[0], ref[1]

    def value(t4):
        return experts.mxfp4_dequantize(t4[0].cpu().numpy(), t4[1].cpu().numpy())

    def quantised(v):
        return experts.mxfp4_dequantize(*experts.mxfp4_quantize(v))

    xv, up, down, hv = d["x_v"], d["up_v"], d["down_v"], host(h)
    if mx:
        xv, up, down, hv = quantised(xv), value(d["up4"]), value(d["down4"]), quantised(hv)
    r, b = _reference(xv, up, d["bu_v"], off, tok, True, hidden)
    check(host(h), r, b, f"up t={t} mxfp4={mx}")
    r, b = _reference(hv, down, d["bd_v"], off, None, False, inner)
    check(host(y), r, b, f"down t={t} mxfp4={mx}")
    r = experts.combine(host(y), ref[2], host(weight))
    acc = (k + 1) * 2.0 ** -23 * experts.combine(np.abs(host(y)), ref[2], host(weight))
    assert np.all(np.abs(host(out) - r) <= acc + 2.0 ** -8 * (np.abs(r) + acc))
    assert sa.sink_attn_device_status(True) == SA_OK


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp4"])
def test_layer_on_streams_and_in_a_graph(mx):
    """Two streams at once, and a captured step replayed on new inputs, give the eager results
    bit for bit."""
    sa = require_gpu()
    a, b = (_layer_inputs(sa, s, 53, 512, 384, 16, 4) for s in (41, 42))
    want = [_layer(sa, d, mx)[-1].clone() for d in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = []
        for d, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                got.append(_layer(sa, d, mx)[-1])
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    x = a["x"].clone()
    step = dict(a, x=x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _layer(sa, step, mx)[-1]
    other = a["x"].flip(0).contiguous()
    want_other = _layer(sa, dict(a, x=other), mx)[-1].clone()
    for src, w in ((a["x"], want[0]), (other, want_other), (a["x"], want[0])):
        x.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    assert sa.sink_attn_device_status(True) == SA_OK
