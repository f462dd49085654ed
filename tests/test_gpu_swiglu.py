"""The SwiGLU of the expert products far from ordinary values, against the formula in fp64:
infinite gates and ups, gates whose sigmoid leaves fp32's range, alpha at both ends of it.

With x = 0 the accumulators are 0 and the bias alone gives gate and up, exactly (a bf16 number
plus 0 in fp32).  What is left is the activation's own arithmetic:

    z = (-alpha g) log2(e): two products and the constant, 3 x 2^-24 of z, which is 3 |alpha g| 2^-24
        of 2^z; 2^z itself by ex2.approx (2^-22), the sum 1 + 2^z (2^-24), its reciprocal by
        rcp.approx (2^-22), two products and the sum u + 1 (3 x 2^-24): together
        (12 + 3 |alpha g|) 2^-24 of the result, to first order; 16 + 4 |alpha g| leaves room for
        the second, as long as |alpha g| 2^-22 is small
    a sigmoid below 2^-126 counts as 0: |g (u + 1)| 2^-126 of the result, with twice that for
        sigmoids around 2^-126
    a product below fp32's normal numbers is off by at most 2^-150, u + 1 times that in the
        result; the last rounding by 2^-8 of it, or 2^-134 below bf16's normal numbers."""
import numpy as np
import pytest
import torch

from gpu_common import dev, host, require_gpu
from oracle import experts

pytestmark = pytest.mark.gpu

INF = float("inf")
# rows: 1 and 40 in one group take single CTAs, 60 a pair; outputs in 16-byte pieces or one by one
FORMS = [(mx, rows, wide) for mx in (False, True) for rows in (1, 60) for wide in (True, False)]


def _activation(sa, gates, ups, alpha, limit, mx, rows, wide):
    """(out [rows, n / 2] of every (gate, up), the same by the formula in fp64, gates, ups)."""
    g, u = (v.reshape(-1) for v in np.meshgrid(gates, ups))
    pad = (-len(g)) % 8 + (0 if wide else 1)   # n / 2 a multiple of 8 or not
    g, u = (np.concatenate([v, np.ones(pad)]) for v in (g, u))
    bias = torch.from_numpy(np.stack([g, u], -1).reshape(1, -1)).to(torch.bfloat16)
    y = bias.double().numpy()
    n, k = y.shape[1], 64
    off = dev(np.array([0, rows], dtype=np.int32))
    if mx:
        zero = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
        operands = (zero(rows, k // 2), zero(rows, 16), zero(1, n, k // 2), zero(1, n, 16))
        out = sa.grouped_mxfp4_linear_swiglu(*operands, off, bias.cuda(), alpha=alpha, limit=limit)
    else:
        x, w = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((rows, k), (1, n, k)))
        out = sa.grouped_linear_swiglu(x, w, off, bias.cuda(), alpha=alpha, limit=limit)
    assert sa.sink_attn_device_status(True) == 0
    with np.errstate(over="ignore", invalid="ignore"):
        ref = experts.swiglu(y, alpha, limit)[0]
        g, u = np.minimum(y[0, 0::2], limit), np.clip(y[0, 1::2], -limit, limit)
    return host(out), ref, g, u


def _check(got, ref, g, u, alpha):
    """Infinities and NaN where the formula has them, everything else within the bound above."""
    top = float(torch.finfo(torch.bfloat16).max)
    for row in got:
        assert np.array_equal(np.isnan(row), np.isnan(ref))
        at = np.isinf(ref)
        assert np.array_equal(row[at], ref[at])
        at = np.isfinite(ref) & (np.abs(ref) < 0.99 * top)   # the rest may round to an infinity
        r, gg, v = ref[at], np.abs(g[at]), np.abs(u[at] + 1.0)
        slope = (16 + 4 * np.minimum(abs(alpha) * gg, 2.0 ** 20)) * 2.0 ** -24
        bound = slope * np.abs(r) + gg * v * 2.0 ** -125 + v * 2.0 ** -150
        bound += 2.0 ** -8 * (np.abs(r) + bound) + 2.0 ** -134
        err = np.abs(row[at] - r)
        assert np.all(err <= bound), (g[at][err > bound], u[at][err > bound], row[at][err > bound], r[err > bound])


@pytest.mark.parametrize("mx,rows,wide", FORMS)
def test_infinite_gates_and_ups(mx, rows, wide):
    """Without a clamp an infinite gate gives an infinity of the sign of u + 1, and NaN only where
    the formula does: u = -1, and gates of minus infinity."""
    sa = require_gpu()
    gates = [INF, -INF, 2.0, -3.0, 0.0]
    ups = [INF, -INF, 0.0, -0.5, -1.0, -1.0078125, -2.0, 5.0, 1e30, -1e30]
    for alpha, limit in ((1.702, INF), (1.702, 7.0), (0.5, 1e20)):
        got, ref, g, u = _activation(sa, gates, ups, alpha, limit, mx, rows, wide)
        _check(got, ref, g, u, alpha)
    got, ref, g, u = _activation(sa, [INF], [0.0, -0.5, -2.0, -1.0], 1.702, INF, mx, rows, wide)
    assert got[0, :3].tolist() == [INF, INF, -INF] and np.isnan(got[0, 3])


@pytest.mark.parametrize("mx,rows,wide", FORMS)
def test_sigmoids_below_the_range_of_fp32(mx, rows, wide):
    """Large negative gates under small and ordinary alpha: what is dropped stays below
    |g (u + 1)| 2^-126, whatever alpha is."""
    sa = require_gpu()
    ups = [0.0, 1.0, -1.0, -3.0, 6.0]
    for alpha, gates in ((1e-30, [-8.8e31, -8.0e31, -1e32, -3e30, 1e31]), (1e-28, [-1e30, -8.6e29, -9e29, 1e30]),
                         (1.702, [-40.0, -51.0, -52.0, -60.0, -88.0, -300.0, -1e30]), (-0.25, [300.0, 340.0, 360.0, 1e4])):
        got, ref, g, u = _activation(sa, gates, ups, alpha, INF, mx, rows, wide)
        _check(got, ref, g, u, alpha)


@pytest.mark.parametrize("mx,rows,wide", FORMS)
def test_alpha_at_the_end_of_its_range(mx, rows, wide):
    """alpha log2(e) does not fit into fp32 although alpha does: gates so small that alpha g is
    around 1 still see their sigmoid, and a gate of 0 gives 0."""
    sa = require_gpu()
    tiny = 2.0 ** -126
    gates = [0.0, -0.0, tiny, -tiny, 1.5 * tiny, -1.5 * tiny, 8 * tiny, -4 * tiny, 1.0, -1.0]
    ups = [2.0 ** 90, -2.0 ** 90, 1.0]
    for alpha in (3.4e38, -3.4e38, 2.3e38, 2.0e38, 1.0):
        got, ref, g, u = _activation(sa, gates, ups, np.float32(alpha).item(), INF, mx, rows, wide)
        _check(got, ref, g, u, alpha)
