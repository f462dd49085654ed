"""Grouped products whose CTAs go round every ring many times: deep K (several staging places
of MXFP4 scales per tile, more of them than there are places), hundreds of tiles, experts of
more than eight row tiles, and ragged ones beside them, against fp64 products on the GPU."""
import numpy as np
import pytest
import torch

from experts_common import check, linear_bound, sizes_to_offsets, swiglu_bound
from gpu_common import dev, host, require_gpu
from oracle import experts

pytestmark = pytest.mark.gpu

ALPHA, LIMIT = 1.702, 7.0
# rows of the experts, features, K: 2880 takes two places of scales per tile of a pair of CTAs,
# 4992 and 5024 four (there are three), 1568 two of which the second holds one block
PAIRS = [([2300, 700, 33, 0, 1900, 225], 5760, 2880), ([1850, 97, 1000, 500, 1], 5140, 4992),
         ([600, 2100, 450], 5760, 5024), ([1000, 2048, 31], 5760, 1568)]
SINGLES = [([3, 40, 64, 1, 0, 17, 30, 48, 5, 9, 33, 2], 5760, 2880), ([1, 2, 0, 1, 1, 2, 1, 2] * 2, 2880, 5024),
           ([45, 12, 60, 38] * 2, 3600, 4992)]


def _bf16(g, shape, std=1.0):
    """(bf16 tensor, its fp64 values)."""
    t = (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)
    return t, t.double()


def _mxfp4(g, shape, std=1.0):
    """(codes, scales, their fp64 values): any code, neighbouring blocks of different scale, so that
    another block's scale would show."""
    k = shape[-1]
    codes = torch.randint(0, 256, (*shape[:-1], k // 2), generator=g, device="cuda", dtype=torch.uint8)
    columns = experts.scale_columns(k)
    scales = torch.full((*shape[:-1], columns), 255, dtype=torch.uint8, device="cuda")  # padding: never used
    power = torch.randint(-2, 2, (*shape[:-1], k // 32), generator=g, device="cuda") + round(np.log2(std / 2.5))
    scales[..., : k // 32] = (power + 127).to(torch.uint8)
    table = torch.from_numpy(experts.E2M1).cuda()
    value = table[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    value.view(*shape[:-1], k // 32, 32).mul_(torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), power).unsqueeze(-1))
    return codes, scales, value


def _check_groups(sa, sizes, n, k, mx, gather, act):
    rng = np.random.default_rng(sum(sizes) + n + k)
    e, start = len(sizes), 2
    offsets = sizes_to_offsets(sizes, start)
    rows = int(offsets[-1]) + 3
    x_rows = 900 if gather else rows
    token = rng.integers(0, x_rows, rows).astype(np.int32) if gather else None
    g = torch.Generator(device="cuda").manual_seed(sum(sizes))
    make = _mxfp4 if mx else _bf16
    *x, xd = make(g, (x_rows, k))
    *w, wd = make(g, (e, n, k), k ** -0.5)
    bias, bd = _bf16(g, (e, n))
    name = ("grouped_mxfp4_linear_" if mx else "grouped_linear_") + ("swiglu" if act else "bias")
    call = lambda: getattr(sa, name)(*x, *w, dev(offsets), bias, row_token=None if token is None else dev(token))  # noqa: E731
    out = call()
    for i in range(e):
        lo, hi = int(offsets[i]), int(offsets[i + 1])
        if lo == hi:
            continue
        xi = xd[lo:hi] if token is None else xd[torch.from_numpy(token[lo:hi]).long().cuda()]
        y = xi @ wd[i].T + bd[i]
        mag = (xi.abs() @ wd[i].abs().T + bd[i].abs()).cpu().numpy()
        if act:
            gate, up = y[:, 0::2].clamp(max=LIMIT), y[:, 1::2].clamp(-LIMIT, LIMIT)
            ref = (gate * torch.sigmoid(ALPHA * gate) * (up + 1)).cpu().numpy()
            bound = swiglu_bound(y.cpu().numpy(), mag, k, ALPHA, LIMIT)
        else:
            ref = y.cpu().numpy()
            bound = linear_bound(ref, mag, k)
        check(host(out[lo:hi]), ref, bound, f"expert {i} of {sizes}, {k} -> {n}, mxfp4={mx}")
    inside = slice(start, int(offsets[-1]))
    for _ in range(3):  # the same bits every time, whatever the schedule
        assert torch.equal(call()[inside], out[inside])
    assert sa.sink_attn_device_status(True) == 0


@pytest.mark.parametrize("act", [False, True], ids=["bias", "swiglu"])
@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gather"])
@pytest.mark.parametrize("case", range(len(PAIRS)))
def test_mxfp4_pairs(case, gather, act):
    _check_groups(require_gpu(), *PAIRS[case], True, gather, act)


@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gather"])
def test_bf16_pairs(gather):
    _check_groups(require_gpu(), *PAIRS[0], False, gather, gather)


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp4"])
@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gather"])
@pytest.mark.parametrize("case", range(len(SINGLES)))
def test_single_ctas(case, gather, mx):
    _check_groups(require_gpu(), *SINGLES[case], mx, gather, case == 0)
