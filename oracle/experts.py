"""fp64 CPU oracle for the expert layer behind the router.  TEST INFRASTRUCTURE ONLY.

Only the tests and the smoke check may use this module.  The library never calls it; it
shares no code with the CUDA path.  Every number is fp64; bf16 inputs are widened exactly.

The page "GPT-OSS on day 0" (Perplexity, 2025) names the pieces: a SwiGLU activation and
bias terms in the experts, weights that ship in MXFP4, a combine by weighted accumulation.
Readings taken where it is silent:

E1. pairs are ordered by expert, and within an expert by (token, slot);
E2. SwiGLU is the clamped form of the public GPT-OSS configuration on interleaved gate
    (even) and up (odd) features: g * sigmoid(alpha g) * (u + 1), g = min(gate, limit),
    u = clamp(up, -limit, limit);
E3. MXFP4 is the OCP MX format (E2M1 in blocks of 32, E8M0 scale) with the conversion of
    that specification: scale 2^(floor(log2 max) - 2), round to nearest even, saturate;
    a block that holds an infinity or a NaN becomes NaN as a whole.
"""
from __future__ import annotations

import numpy as np

__all__ = ["group_rows", "grouped_linear", "swiglu", "combine", "mxfp4_quantize", "mxfp4_dequantize",
           "scale_columns", "E2M1"]

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


def group_rows(topk_idx, num_experts: int):
    """(expert_offsets [E + 1], row_token [T * k], pair_row [T, k]), reading E1; indices
    outside [0, E) have no row."""
    idx = np.asarray(topk_idx)
    t, k = idx.shape
    rows = [[] for _ in range(num_experts)]
    for p, e in enumerate(idx.reshape(-1).tolist()):
        if 0 <= e < num_experts:
            rows[e].append(p)
    offsets = np.zeros(num_experts + 1, dtype=np.int32)
    offsets[1:] = np.cumsum([len(r) for r in rows])
    row_token = np.full(t * k, -1, dtype=np.int32)
    pair_row = np.full(t * k, -1, dtype=np.int32)
    for r, p in enumerate([p for group in rows for p in group]):
        row_token[r] = p // k
        pair_row[p] = r
    return offsets, row_token, pair_row.reshape(t, k)


def grouped_linear(x, w, bias, offsets, row_token=None):
    """x [X, K], w [E, N, K], bias [E, N] or None, all fp64 -> (y [R, N], magnitude [R, N]),
    NaN outside the groups.  ``magnitude`` is sum |x w| + |bias|, for error bounds."""
    r = x.shape[0] if row_token is None else len(row_token)
    y = np.full((r, w.shape[1]), np.nan)
    mag = np.full_like(y, np.nan)
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo == hi:
            continue
        xs = x[lo:hi] if row_token is None else x[np.asarray(row_token[lo:hi])]
        y[lo:hi] = xs @ w[e].T
        mag[lo:hi] = np.abs(xs) @ np.abs(w[e]).T
        if bias is not None:
            y[lo:hi] += bias[e]
            mag[lo:hi] += np.abs(bias[e])
    return y, mag


def swiglu(y, alpha: float, limit: float):
    """Reading E2 on the last dimension."""
    g = np.minimum(y[..., 0::2], limit)
    u = np.clip(y[..., 1::2], -limit, limit)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-alpha * g)) * (u + 1.0)


def combine(y, pair_row, weight):
    """out[t] = sum_r weight[t, r] y[pair_row[t, r]]; -1 adds nothing."""
    out = np.zeros((pair_row.shape[0], y.shape[1]))
    for r in range(pair_row.shape[1]):
        has = pair_row[:, r] >= 0
        out[has] += weight[has, r][:, None] * y[pair_row[has, r]]
    return out


def scale_columns(k: int) -> int:
    return -(-(k // 32) // 16) * 16


def mxfp4_quantize(x):
    """x [R, K] fp64 -> (codes uint8 [R, K / 2], scales uint8 [R, scale_columns(K)])."""
    x = np.asarray(x, dtype=np.float64)
    r, k = x.shape
    blocks = x.reshape(r, k // 32, 32)
    largest = np.abs(blocks).max(-1)
    ok = np.isfinite(largest)
    _, e = np.frexp(np.where(ok & (largest > 0), largest, 1.0))  # largest in [2^(e-1), 2^e)
    e = np.where(largest > 0, e - 1 - 2, -127).clip(-127, 127)
    v = np.where(ok[..., None], np.ldexp(np.where(ok[..., None], blocks, 0.0), -e[..., None]), 0.0)
    # nearest magnitude, ties to the even code (even codes listed first win ties)
    order = [0, 2, 4, 6, 1, 3, 5, 7]
    away = np.abs(np.abs(v)[..., None] - E2M1[order])
    code = np.array(order)[away.argmin(-1)] + 8 * np.signbit(v)
    code = np.where(ok[..., None], code, 0).astype(np.uint8).reshape(r, k)
    scales = np.zeros((r, scale_columns(k)), dtype=np.uint8)
    scales[:, : k // 32] = np.where(ok, e + 127, 255)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def mxfp4_dequantize(codes, scales):
    """The fp64 values of codes [..., K / 2] and scales [..., >= K / 32]."""
    k = 2 * codes.shape[-1]
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], k)
    s = np.asarray(scales)[..., : k // 32].astype(np.int64)
    power = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return E2M1[nib] * np.repeat(power, 32, axis=-1)
