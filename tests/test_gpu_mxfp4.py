"""GPU parity of the MXFP4 conversions: codes and scales equal the fp64 oracle's bit for bit
(scaling by a power of two is exact, so the only rounding is the one to E2M1)."""
import numpy as np
import pytest
import torch

from gpu_common import require_gpu
from oracle import experts

pytestmark = pytest.mark.gpu


def _same(sa, x):
    """Codes and scales of x [R, K] against the oracle's."""
    codes, scales = sa.mxfp4_quantize(x)
    rc, rs = experts.mxfp4_quantize(x.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)
    return codes, scales


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("r,k", [(1, 32), (3, 64), (64, 2880), (129, 512), (1000, 544), (7, 4128)])
def test_quantize_normal_values(r, k, dtype):
    sa = require_gpu()
    g = torch.Generator().manual_seed(r * k)
    x = torch.randn(r, k, generator=g) * torch.exp(4 * torch.randn(r, k // 32, generator=g)).repeat_interleave(32, 1)
    x[torch.rand(r, k, generator=g) < 0.05] = 0
    x = x.to(dtype).cuda()
    codes, scales = _same(sa, x)
    value = sa.mxfp4_dequantize(codes, scales).double().cpu().numpy()
    assert np.array_equal(value, experts.mxfp4_dequantize(codes.cpu().numpy(), scales.cpu().numpy()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_ties_and_neighbours(dtype):
    """Every midpoint between two E2M1 values, and the nearest representable values beside it,
    in blocks whose largest value is 4, 6 or just below 8, at scales over the whole range."""
    sa = require_gpu()
    eps = torch.finfo(dtype).eps
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0])
    v = torch.cat([mid, mid * (1 + eps), mid * (1 - eps / 2)])
    v = torch.cat([v, -v])                       # 54 values in two blocks of 27 + the largest
    blocks = []
    for top in (4.0, 6.0, 7.96875):
        for part in v.clamp(-top, top).split(27):
            blocks.append(torch.cat([part, torch.tensor([top, -0.0, 0.0, 0.5, 1.0])]))
    base = torch.stack(blocks)
    for power in (-126, -120, -60, -3, 0, 5, 90, 124):
        x = (base.double() * 2.0 ** power).to(dtype).cuda()
        _same(sa, x)


def test_quantize_extremes():
    """Zeros, subnormal numbers, the largest numbers, infinities and NaN; only the block that
    holds a value that is not finite becomes NaN."""
    sa = require_gpu()
    for dtype in (torch.bfloat16, torch.float32):
        f = torch.finfo(dtype)
        x = torch.zeros(9, 96, dtype=dtype)
        x[1] = f.max
        x[2, :32], x[2, 32:64], x[2, 64:] = f.tiny, f.tiny / 2, -f.smallest_normal * f.eps
        x[3, 5], x[4, 40], x[5, 70] = float("inf"), float("-inf"), float("nan")
        x[6] = -0.0
        x[7] = torch.linspace(-1, 1, 96).to(dtype) * f.tiny * 8
        x[8] = torch.linspace(-f.max, f.max, 96, dtype=torch.float64).to(dtype)
        codes, scales = _same(sa, x.cuda())
        value = sa.mxfp4_dequantize(codes, scales)
        nan = torch.zeros(9, 96, dtype=torch.bool)
        nan[3, :32], nan[4, 32:64], nan[5, 64:] = True, True, True
        assert torch.equal(torch.isnan(value).cpu(), nan)


def test_dequantize_every_code_under_every_scale():
    sa = require_gpu()
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (1, 1))  # K = 32: all pairs of codes
    codes = np.tile(codes, (256, 1))
    scales = np.zeros((16 * 256, 16), dtype=np.uint8)
    scales[:, 0] = np.repeat(np.arange(256), 16)
    scales[:, 1:] = 255
    got = sa.mxfp4_dequantize(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    ref = torch.from_numpy(experts.mxfp4_dequantize(codes, scales)).to(torch.bfloat16)  # beyond bf16: infinite
    assert torch.equal(torch.isnan(got).cpu(), torch.isnan(ref))
    assert torch.equal(torch.nan_to_num(got.cpu(), nan=1.0), torch.nan_to_num(ref, nan=1.0))


def test_shapes_and_given_outputs():
    sa = require_gpu()
    x = torch.randn(3, 5, 192, dtype=torch.bfloat16, device="cuda")
    codes, scales = sa.mxfp4_quantize(x)
    assert codes.shape == (3, 5, 96) and scales.shape == (3, 5, 16)
    assert (scales[..., 6:] == 0).all()
    c2, s2 = torch.full_like(codes, 9), torch.full_like(scales, 9)
    sa.mxfp4_quantize(x, codes=c2, scales=s2)
    assert torch.equal(c2, codes) and torch.equal(s2, scales)
    flat = sa.mxfp4_quantize(x.view(15, 192))
    assert torch.equal(flat[0].view_as(codes), codes) and torch.equal(flat[1].view_as(scales), scales)
    out = torch.empty(3, 5, 192, dtype=torch.bfloat16, device="cuda")
    assert sa.mxfp4_dequantize(codes, scales, out=out) is out
    empty = sa.mxfp4_quantize(x[:0])
    assert empty[0].shape == (0, 5, 96) and sa.mxfp4_dequantize(*empty).shape == (0, 5, 192)
    one = sa.mxfp4_quantize(x[0, 0])
    assert torch.equal(one[0], codes[0, 0]) and torch.equal(one[1], scales[0, 0])
