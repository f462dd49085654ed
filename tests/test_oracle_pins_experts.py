"""The expert-layer oracle against hand-worked values, brute force and identities (CPU)."""
import numpy as np
import pytest
import torch

from oracle import experts


def test_group_rows_by_hand():
    idx = np.array([[2, 0], [0, 2], [-1, 2], [1, 1]])
    off, tok, row = experts.group_rows(idx, 4)
    assert off.tolist() == [0, 2, 4, 7, 7]
    assert tok.tolist() == [0, 1, 3, 3, 0, 1, 2, -1]
    assert row.tolist() == [[4, 0], [1, 5], [-1, 6], [2, 3]]


@pytest.mark.parametrize("seed", range(4))
def test_group_rows_is_a_stable_sort(seed):
    rng = np.random.default_rng(seed)
    t, k, e = 50, 3, 7
    idx = rng.integers(-1, e + 1, (t, k))          # -1 and e: no expert
    off, tok, row = experts.group_rows(idx, e)
    flat = idx.reshape(-1)
    has = (flat >= 0) & (flat < e)
    order = np.argsort(np.where(has, flat, e), kind="stable")[: has.sum()]
    assert np.array_equal(tok[: len(order)], order // k) and (tok[len(order):] == -1).all()
    assert np.array_equal(row.reshape(-1)[order], np.arange(len(order))) and (row.reshape(-1)[~has] == -1).all()
    assert np.array_equal(np.diff(off), [np.sum(flat == i) for i in range(e)])


def test_swiglu_by_hand():
    # g = 0 -> 0; alpha 0 -> sigmoid 1/2; clamps: g from above only, u from both sides
    y = np.array([[0.0, 5.0], [2.0, 3.0], [9.0, 9.0], [-9.0, -9.0]])
    out = experts.swiglu(y, 0.0, 7.0)
    assert out.reshape(-1).tolist() == [0.0, 2.0 / 2 * 4, 7.0 / 2 * 8, -9.0 / 2 * -6]
    y = np.random.default_rng(0).standard_normal((5, 8)) * 4
    t = torch.from_numpy(y)
    g, u = t[:, 0::2].clamp(max=1.5), t[:, 1::2].clamp(-1.5, 1.5)
    assert np.allclose(experts.swiglu(y, 1.702, 1.5), (g * torch.sigmoid(1.702 * g) * (u + 1)).numpy(), rtol=1e-14, atol=0)


def test_grouped_linear_is_a_loop_over_rows():
    rng = np.random.default_rng(1)
    x, w, b = rng.standard_normal((6, 5)), rng.standard_normal((3, 4, 5)), rng.standard_normal((3, 4))
    off, tok = np.array([1, 3, 3, 6]), np.array([0, 5, 5, 2, 1, 0, 3])
    y, mag = experts.grouped_linear(x, w, b, off, tok)
    assert np.isnan(y[[0, 6]]).all()
    for r, e in ((1, 0), (2, 0), (3, 2), (4, 2), (5, 2)):
        for n in range(4):
            assert np.isclose(y[r, n], sum(x[tok[r], i] * w[e, n, i] for i in range(5)) + b[e, n], rtol=1e-13)
            assert mag[r, n] >= abs(y[r, n]) - 1e-12


def test_combine_by_hand():
    y = np.array([[1.0, 2.0], [10.0, 20.0], [np.nan, np.nan]])
    out = experts.combine(y, np.array([[1, 0], [-1, 1], [-1, -1]]), np.array([[0.5, 2.0], [9.0, 0.25], [1.0, 1.0]]))
    assert out.tolist() == [[7.0, 14.0], [2.5, 5.0], [0.0, 0.0]]


def test_mxfp4_by_hand():
    x = np.zeros((1, 32))
    x[0, :8] = [6.0, -6.0, 0.25, 0.75, 2.5, 5.0, 0.26, -1.75]   # largest 6: scale 2^0; ties to even
    codes, scales = experts.mxfp4_quantize(x)
    assert scales[0, 0] == 127 and scales.shape == (1, 16) and (scales[0, 1:] == 0).all()
    assert experts.mxfp4_dequantize(codes, scales)[0, :8].tolist() == [6, -6, 0, 1, 2, 4, 0.5, -2]
    assert codes[0, :4].tolist() == [7 | 15 << 4, 0 | 2 << 4, 4 | 6 << 4, 1 | 12 << 4]
    x[0, 0] = 7.9                                               # scale still 1: saturates at 6
    assert experts.mxfp4_dequantize(*experts.mxfp4_quantize(x))[0, 0] == 6
    x[0, 0] = 8.0                                               # scale 2: exact
    codes, scales = experts.mxfp4_quantize(x)
    assert scales[0, 0] == 128 and experts.mxfp4_dequantize(codes, scales)[0, 0] == 8


def test_mxfp4_nearest_of_all_and_idempotent():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((20, 64)) * np.exp(3 * rng.standard_normal((20, 1)))
    codes, scales = experts.mxfp4_quantize(x)
    v = experts.mxfp4_dequantize(codes, scales)
    s = np.repeat(np.ldexp(1.0, scales[:, :2].astype(int) - 127), 32, axis=1)
    best = np.abs(x[..., None] - experts.E2M1 * s[..., None]).min(-1)
    assert np.array_equal(np.abs(x - v), best)
    assert np.all(np.abs(x).reshape(20, 2, 32).max(-1) < 8 * np.ldexp(1.0, scales[:, :2].astype(int) - 127))
    again = experts.mxfp4_quantize(v)   # a value's own block maximum is at least 4 scales: same scale
    assert np.array_equal(again[0] & 0x77, codes & 0x77) and np.array_equal(again[1], scales)


def test_mxfp4_blocks_that_are_not_finite():
    x = np.ones((2, 64))
    x[0, 3], x[1, 40] = np.inf, np.nan
    codes, scales = experts.mxfp4_quantize(x)
    assert scales[:, :2].tolist() == [[255, 125], [125, 255]]
    assert np.isnan(experts.mxfp4_dequantize(codes, scales)).reshape(2, 2, 32).all(-1).tolist() == [[True, False], [False, True]]
