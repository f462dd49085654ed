"""Inputs and error bounds shared by the expert-layer GPU tests.

Bounds, from the arithmetic.  bf16 x bf16 products, and E2M1 products times powers of two,
are exact in fp32; the tensor core sums K of them in fp32, which (for recursive summation,
allowing truncation instead of rounding) errs by at most K 2^-23 sum |x w|; the bias adds one
fp32 rounding of the result.  ``acc`` below is that bound with the bias among the K + 1 terms.
The bf16 result adds half a step: 2^-8 of its magnitude.

SwiGLU out = f(g) (u + 1), f(g) = g sigmoid(alpha g): |f'| <= 1.1 for every alpha, and the
clamps never enlarge a difference, so errors acc_g, acc_u of its arguments change it by at
most 1.1 acc_g |u + 1| + |f(g)| acc_u + 1.1 acc_g acc_u.  Its evaluation in fp32 adds a
relative error: the CUDA guide bounds __expf by 2 + 1.173 |x| units in the last place and
__fdividef by 2, and the two sums and two products round once each, so (16 + 2 |alpha g|) 2^-23
covers it.  Where exp(-alpha g) overflows the result is 0 and the value below 1e-30."""
import numpy as np
import torch

from oracle import experts


def sizes_to_offsets(sizes, start=0):
    return np.concatenate([[start], start + np.cumsum(sizes)]).astype(np.int32)


def bf16_normal(rng, shape, std=1.0):
    """(bf16 CUDA tensor, its fp64 values)."""
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * np.float32(std)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def mxfp4_normal(rng, shape, std=1.0):
    """(codes, scales) CUDA tensors of a quantised normal matrix, and its fp64 values."""
    x = rng.standard_normal((int(np.prod(shape[:-1])), shape[-1])) * std
    codes, scales = experts.mxfp4_quantize(x)
    value = experts.mxfp4_dequantize(codes, scales).reshape(shape)
    scales[:, shape[-1] // 32:] = 255  # padding bytes: never used, whatever they hold
    return (torch.from_numpy(codes.reshape(*shape[:-1], codes.shape[-1])).cuda(),
            torch.from_numpy(scales.reshape(*shape[:-1], scales.shape[-1])).cuda(), value)


def acc_bound(mag, k):
    return (k + 1) * 2.0 ** -23 * mag


def linear_bound(ref, mag, k):
    acc = acc_bound(mag, k)
    return acc + 2.0 ** -8 * (np.abs(ref) + acc)


def swiglu_bound(y, mag, k, alpha, limit):
    acc = acc_bound(mag, k)
    ag, au = acc[..., 0::2], acc[..., 1::2]
    g = np.minimum(y[..., 0::2], limit)
    u = np.clip(y[..., 1::2], -limit, limit)
    with np.errstate(over="ignore"):
        f = np.abs(g / (1.0 + np.exp(-alpha * g)))
    ref = f * np.abs(u + 1.0)
    err = 1.1 * ag * np.abs(u + 1.0) + f * au + 1.1 * ag * au + (16 + 2 * abs(alpha) * np.abs(g)) * 2.0 ** -23 * ref
    return err + 2.0 ** -8 * (ref + err) + 1e-30


def check(got, ref, bound, what):
    """Every element of the groups within its bound, and the RMS error below 2^-8 of the RMS
    result (a dropped K step or a shifted tile fails that even where the bound is loose)."""
    got, inside = np.asarray(got, dtype=np.float64), ~np.isnan(ref)
    if not inside.any():  # an expert without rows
        return
    err = np.abs(got[inside] - ref[inside])
    assert np.isfinite(err).all(), f"{what}: {np.sum(~np.isfinite(err))} results are not finite"
    rms, rms_ref = np.sqrt(np.mean(err ** 2)), np.sqrt(np.mean(ref[inside] ** 2))
    print(f"ERR {what}: max {err.max():.3e} rms {rms:.3e} (rms out {rms_ref:.3e})")
    assert np.all(err <= bound[inside]), f"{what}: {np.max(err - bound[inside])} beyond the bound"
    assert rms <= 2.0 ** -8 * rms_ref, f"{what}: rms error {rms} of {rms_ref}"
