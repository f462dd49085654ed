"""GQA attention with per-head softmax sinks on GB300 (sm_103a).

Thin ctypes binding of ``libsinkattn.so`` (C ABI in ``include/sink_attn.h``).
Every function below only marshals arguments: it reads shapes off the torch
tensors, allocates outputs when none are given, passes raw device pointers
and the current CUDA stream, and turns a non-zero status into an exception.
All arithmetic runs in the library's CUDA kernels; there is no fallback.

The operation (page "GPT-OSS on day 0", section "Kernels for GPT-OSS / Sink
Attention"): ``attn = softmax(q k^T * sm_scale + sink) V`` where each query
head's sink is one extra softmax logit that carries no value row.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

__all__ = [
    "SinkAttnError", "library_path", "load_library", "sink_attn_prefill", "sink_attn_prefill_paged",
    "sink_attn_decode", "sink_attn_merge", "sink_attn_decode_splits", "sink_attn_device_status",
    "sink_attn_set_wait_timeout_ns", "sink_attn_status_string", "sink_attn_abi_version",
    "sink_attn_selftest_wait_timeout", "sink_attn_decode_noalloc", "moe_router_topk_softmax",
    "qkv_bias_rope", "qkv_bias_rope_append_paged", "linear_bias", "moe_router", "GPT_OSS_YARN",
    "EXPORTED_SYMBOLS", "qkv_bias_rope_kv", "qkv_bias_rope_append_paged_kv", "sink_attn_prefill_qkv",
    "sink_attn_prefill_paged_qkv", "sink_attn_decode_qkv", "moe_group_rows", "moe_combine",
    "grouped_linear_bias", "grouped_linear_swiglu", "mxfp4_quantize", "mxfp4_dequantize",
    "mxfp4_linear_bias", "grouped_mxfp4_linear_bias", "grouped_mxfp4_linear_swiglu",
    "mxfp4_scale_columns", "GPT_OSS_SWIGLU", "sink_attn_decode_shared", "sink_attn_decode_shared_splits",
    "lora_linear_bias", "lora_workspace_bytes", "moe_router_scores",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libsinkattn.so")
_lib = None

EXPORTED_SYMBOLS = (
    "sink_attn_prefill", "sink_attn_prefill_paged", "sink_attn_decode", "sink_attn_merge",
    "sink_attn_decode_splits", "sink_attn_device_status", "sink_attn_set_wait_timeout_ns",
    "sink_attn_status_string", "sink_attn_abi_version", "sink_attn_selftest_wait_timeout",
    "sink_attn_decode_noalloc", "moe_router_topk_softmax", "qkv_bias_rope",
    "qkv_bias_rope_append_paged", "linear_bias", "moe_router", "qkv_bias_rope_kv",
    "qkv_bias_rope_append_paged_kv", "sink_attn_prefill_qkv", "sink_attn_prefill_paged_qkv",
    "sink_attn_decode_qkv", "moe_group_rows", "moe_combine",
    "grouped_linear_bias", "grouped_linear_swiglu", "mxfp4_quantize", "mxfp4_dequantize",
    "mxfp4_linear_bias", "grouped_mxfp4_linear_bias", "grouped_mxfp4_linear_swiglu",
    "sink_attn_decode_shared", "sink_attn_decode_shared_splits", "lora_linear_bias", "lora_workspace_bytes",
    "moe_router_scores",
)

_p, _i, _f, _d, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_double, ctypes.c_longlong
_SIGNATURES = {
    "sink_attn_prefill": (_i, [_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _f, _i, _p, _p, _p]),
    "sink_attn_prefill_paged": (_i, [_p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i,
                                     _f, _i, _p, _p, _p]),
    "sink_attn_decode": (_i, [_p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _f, _i, _p, _p, _p]),
    "sink_attn_merge": (_i, [_p, _p, _i, _i, _i, _i, _p, _p, _p]),
    "sink_attn_decode_splits": (_i, [_i, _i, _i, _i, _i]),
    "sink_attn_device_status": (_i, [_i]),
    "sink_attn_set_wait_timeout_ns": (None, [ctypes.c_ulonglong]),
    "sink_attn_status_string": (ctypes.c_char_p, [_i]),
    "sink_attn_abi_version": (_i, []),
    "sink_attn_selftest_wait_timeout": (_i, [ctypes.c_ulonglong, _p]),
    "sink_attn_decode_noalloc": (_i, [_p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _f, _i, _p, _p,
                                      _p]),
    "moe_router_topk_softmax": (_i, [_p, _ll, _i, _i, _p, _p, _p, _p]),
    "linear_bias": (_i, [_p, _p, _p, _i, _i, _i, _p, _p]),
    "moe_router": (_i, [_p, _p, _p, _i, _i, _i, _i, _p, _p, _p, _p]),
    "qkv_bias_rope": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _i, _d, _d, _i, _d, _d, _p, _p, _p, _p]),
    "qkv_bias_rope_append_paged": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _i, _d, _d, _i, _d, _d, _p, _p,
                                        _p, _p, _i, _i, _i, _p]),
    "qkv_bias_rope_kv": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _i, _d, _d, _i, _d, _d, _p, _p, _p, _p]),
    "qkv_bias_rope_append_paged_kv": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _i, _d, _d, _i, _d, _d, _p, _p,
                                           _p, _i, _i, _i, _p, _p]),
    "sink_attn_prefill_qkv": (_i, [_p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _f, _i, _p, _p, _p]),
    "sink_attn_prefill_paged_qkv": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i,
                                         _i, _f, _i, _p, _p, _p]),
    "sink_attn_decode_qkv": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _f, _i, _p, _p,
                                  _p]),
    "moe_group_rows": (_i, [_p, _i, _i, _i, _p, _p, _p, _p]),
    "moe_combine": (_i, [_p, _p, _p, _i, _i, _i, _i, _p, _p]),
    "grouped_linear_bias": (_i, [_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _p, _p]),
    "grouped_linear_swiglu": (_i, [_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _f, _f, _p, _p]),
    "mxfp4_quantize": (_i, [_p, _i, _ll, _i, _p, _p, _p]),
    "mxfp4_dequantize": (_i, [_p, _p, _ll, _i, _p, _p]),
    "mxfp4_linear_bias": (_i, [_p, _p, _p, _p, _p, _i, _i, _i, _p, _p]),
    "grouped_mxfp4_linear_bias": (_i, [_p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _p, _p]),
    "sink_attn_decode_shared": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i, _f, _i, _i,
                                     _p, _p, _p, _p, _p]),
    "sink_attn_decode_shared_splits": (None, [_i, _i, _i, _i, _i, _i, _i, _p, _p]),
    "lora_linear_bias": (_i, [_p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _p, _p, _p]),
    "lora_workspace_bytes": (None, [_i, _i, _i, _p]),
    "moe_router_scores": (_i, [_p, _i, _ll, _i, _i, _i, _p, _i, _i, _i, _f, _p, _p, _p, _p]),
    "grouped_mxfp4_linear_swiglu": (_i, [_p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _f, _f, _p, _p]),
}

# YaRN constants of the public GPT-OSS model configuration (the pages name YaRN
# but give no constants): rotary base, scale factor, original context length,
# beta_fast, beta_slow.
GPT_OSS_YARN = dict(rope_base=150000.0, factor=32.0, orig_len=4096, beta_fast=32.0, beta_slow=1.0)


class SinkAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({_status_text(status)})")


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libsinkattn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build it with "
                "`python -m attention_softmax_sinks_gb300._build` (nvcc, sm_103a)")
        lib = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _status_text(status: int) -> str:
    try:
        return load_library().sink_attn_status_string(status).decode()
    except Exception:  # library missing: still produce a message
        return "unknown"


def _check(status: int, where: str):
    if status != 0:
        raise SinkAttnError(status, where)


def _ptr(t):
    """Raw device address (ctypes passes Python ints as void*), or None."""
    return None if t is None else t.data_ptr()


def _dev(t, name, dtype):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _out(t, name, dtype, shape, dev):
    """A caller-supplied output: on device index ``dev``, of ``dtype``, contiguous and ``shape``."""
    _dev(t, name, dtype)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the inputs on cuda:{dev}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _same_device(dev, *named):
    """Every (name, tensor) pair with a tensor lies on device index ``dev``."""
    for name, t in named:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, expected cuda:{dev} "
                             "(the device of the first input)")


def _call(fn, dev, stream, *args):
    """fn(*args, stream) with device ``dev`` current for the call and ``stream`` (default: that
    device's current stream) as the last argument; the previous current device is restored."""
    if stream is not None and stream.device_index != dev:
        raise ValueError(f"stream is on cuda:{stream.device_index}, the tensors on cuda:{dev}")
    # the raw handle: a Stream object costs more than the rest of the call
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:  # the tensors are there: CUDA is initialised
        return fn(*args, s)
    with torch.cuda.device(dev):
        return fn(*args, s)


# ----------------------------------------------------------------------------- entry points
def _checked(named):
    """Validate (name, tensor, dtype) triples: CUDA, dtype, contiguous.  Returns the first
    tensor's device and device index."""
    for name, t, dt in named:
        _dev(t, name, dt)
    first = named[0][1]
    return first.device, first.get_device()


def sink_attn_prefill(q, k, v, sinks, cu_seqlens, max_seqlen: int, sm_scale: float,
                      causal: bool = True, out=None, lse=None, return_lse: bool = True,
                      stream=None):
    """Prefill over contiguous ragged sequences (q_len == kv_len).

    q [T, Hq, 64] bf16, k/v [T, Hkv, 64] bf16, sinks [Hq] fp32, cu_seqlens [B+1] int32.
    Returns (out [T, Hq, 64] bf16, lse [T, Hq] fp32 or None).
    """
    dev, di = _checked((("q", q, torch.bfloat16), ("k", k, torch.bfloat16), ("v", v, torch.bfloat16),
                        ("sinks", sinks, torch.float32), ("cu_seqlens", cu_seqlens, torch.int32)))
    t, hq, d = q.shape
    hkv = k.shape[1]
    if k.shape != (t, hkv, d) or v.shape != k.shape:
        raise ValueError("k and v must be [T, Hkv, D] with q's T and D")
    _same_device(di, ("k", k), ("v", v), ("sinks", sinks), ("cu_seqlens", cu_seqlens))
    out = torch.empty_like(q) if out is None else _out(out, "out", torch.bfloat16, q.shape, di)
    if lse is None and return_lse:
        lse = torch.empty((t, hq), dtype=torch.float32, device=dev)
    elif lse is not None:
        _out(lse, "lse", torch.float32, (t, hq), di)
    st = _call(load_library().sink_attn_prefill, di, stream,
               _ptr(q), _ptr(k), _ptr(v), _ptr(sinks), _ptr(cu_seqlens), cu_seqlens.numel() - 1, t,
               int(max_seqlen), hq, hkv, d, float(sm_scale), int(bool(causal)), _ptr(out), _ptr(lse))
    _check(st, "sink_attn_prefill")
    return out, lse


def sink_attn_prefill_paged(q, paged_k, paged_v, page_table, cu_seqlens_q, kv_lens, sinks,
                            max_q_len: int, sm_scale: float, causal: bool = True, out=None,
                            lse=None, return_lse: bool = True, stream=None):
    """New tokens of a mixed batch against a paged cache (bottom-right causal).

    q [Tq, Hq, 64] bf16, paged_k/v [P, Hkv, 16, 64] bf16, page_table [B, max_pages] int32,
    cu_seqlens_q [B+1] int32, kv_lens [B] int32, sinks [Hq] fp32.
    """
    dev, di = _checked((("q", q, torch.bfloat16), ("paged_k", paged_k, torch.bfloat16),
                        ("paged_v", paged_v, torch.bfloat16), ("page_table", page_table, torch.int32),
                        ("cu_seqlens_q", cu_seqlens_q, torch.int32), ("kv_lens", kv_lens, torch.int32),
                        ("sinks", sinks, torch.float32)))
    t, hq, d = q.shape
    num_pages, hkv, page_size, _ = paged_k.shape
    _same_device(di, ("paged_k", paged_k), ("paged_v", paged_v), ("page_table", page_table),
                 ("cu_seqlens_q", cu_seqlens_q), ("kv_lens", kv_lens), ("sinks", sinks))
    out = torch.empty_like(q) if out is None else _out(out, "out", torch.bfloat16, q.shape, di)
    if lse is None and return_lse:
        lse = torch.empty((t, hq), dtype=torch.float32, device=dev)
    elif lse is not None:
        _out(lse, "lse", torch.float32, (t, hq), di)
    st = _call(load_library().sink_attn_prefill_paged, di, stream,
               _ptr(q), _ptr(paged_k), _ptr(paged_v), _ptr(page_table), _ptr(cu_seqlens_q), _ptr(kv_lens),
               _ptr(sinks), cu_seqlens_q.numel() - 1, t, int(max_q_len), hq, hkv, d, page_size,
               page_table.shape[1], num_pages, float(sm_scale), int(bool(causal)), _ptr(out), _ptr(lse))
    _check(st, "sink_attn_prefill_paged")
    return out, lse


def _decode_outputs(out, lse, return_lse, b, s, hq, d, dev, di):
    out_shape, out_dtype = ((b, hq, d), torch.bfloat16) if s == 1 else ((b, s, hq, d), torch.float32)
    lse_shape = (b, hq) if s == 1 else (b, s, hq)
    if out is None:
        out = torch.empty(out_shape, dtype=out_dtype, device=dev)
    else:
        _out(out, "out", out_dtype, out_shape, di)
    if lse is None and (return_lse or s > 1):
        lse = torch.empty(lse_shape, dtype=torch.float32, device=dev)
    elif lse is not None:
        _out(lse, "lse", torch.float32, lse_shape, di)
    return out, lse


def sink_attn_decode(q, paged_k, paged_v, page_table, kv_lens, sinks, sm_scale: float,
                     num_splits: int = 1, out=None, lse=None, return_lse: bool = True, stream=None):
    """One new token per sequence against a paged cache.

    num_splits == 1: returns (out [B, Hq, 64] bf16, lse [B, Hq] fp32).
    num_splits > 1: returns the partials (o [B, S, Hq, 64] fp32, lse [B, S, Hq] fp32)
    for sink_attn_merge.
    """
    dev, di = _checked((("q", q, torch.bfloat16), ("paged_k", paged_k, torch.bfloat16),
                        ("paged_v", paged_v, torch.bfloat16), ("page_table", page_table, torch.int32),
                        ("kv_lens", kv_lens, torch.int32), ("sinks", sinks, torch.float32)))
    b, hq, d = q.shape
    num_pages, hkv, page_size, _ = paged_k.shape
    _same_device(di, ("paged_k", paged_k), ("paged_v", paged_v), ("page_table", page_table),
                 ("kv_lens", kv_lens), ("sinks", sinks))
    s = int(num_splits)
    out, lse = _decode_outputs(out, lse, return_lse, b, s, hq, d, dev, di)
    st = _call(load_library().sink_attn_decode, di, stream,
               _ptr(q), _ptr(paged_k), _ptr(paged_v), _ptr(page_table), _ptr(kv_lens), _ptr(sinks), b, hq,
               hkv, d, page_size, page_table.shape[1], num_pages, float(sm_scale), s, _ptr(out), _ptr(lse))
    _check(st, "sink_attn_decode")
    return out, lse


def sink_attn_decode_noalloc(q, paged_k, paged_v, page_table, kv_lens, sinks, sm_scale: float,
                             num_splits: int, out=None, lse=None, return_lse: bool = True,
                             stream=None):
    """Split decode + merge in one library call that allocates no device memory.

    For callers that cannot allocate when they enqueue work: the split partials
    live in the library's fixed 8 MiB device array (batch * num_splits * Hq * 65
    floats at most).  Pass preallocated ``out`` [B, Hq, 64] bf16 and ``lse``
    [B, Hq] fp32 to keep this wrapper allocation-free as well.  Calls that
    overlap on the GPU race on the shared array.
    """
    dev, di = _checked((("q", q, torch.bfloat16), ("paged_k", paged_k, torch.bfloat16),
                        ("paged_v", paged_v, torch.bfloat16), ("page_table", page_table, torch.int32),
                        ("kv_lens", kv_lens, torch.int32), ("sinks", sinks, torch.float32)))
    b, hq, d = q.shape
    num_pages, hkv, page_size, _ = paged_k.shape
    _same_device(di, ("paged_k", paged_k), ("paged_v", paged_v), ("page_table", page_table),
                 ("kv_lens", kv_lens), ("sinks", sinks))
    out, lse = _decode_outputs(out, lse, return_lse, b, 1, hq, d, dev, di)
    st = _call(load_library().sink_attn_decode_noalloc, di, stream,
               _ptr(q), _ptr(paged_k), _ptr(paged_v), _ptr(page_table), _ptr(kv_lens), _ptr(sinks), b, hq,
               hkv, d, page_size, page_table.shape[1], num_pages, float(sm_scale), int(num_splits),
               _ptr(out), _ptr(lse))
    _check(st, "sink_attn_decode_noalloc")
    return out, lse


def sink_attn_merge(partial_o, partial_lse, out=None, lse=None, return_lse: bool = True,
                    stream=None):
    """Merge split partials o [B, S, H, 64] fp32 / lse [B, S, H] fp32 -> (out bf16, lse fp32)."""
    dev, di = _checked((("partial_o", partial_o, torch.float32), ("partial_lse", partial_lse, torch.float32)))
    b, s, h, d = partial_o.shape
    if tuple(partial_lse.shape) != (b, s, h):
        raise ValueError(f"partial_lse must be {(b, s, h)}, got {tuple(partial_lse.shape)}")
    _same_device(di, ("partial_lse", partial_lse))
    out = (torch.empty((b, h, d), dtype=torch.bfloat16, device=dev) if out is None
           else _out(out, "out", torch.bfloat16, (b, h, d), di))
    if lse is None and return_lse:
        lse = torch.empty((b, h), dtype=torch.float32, device=dev)
    elif lse is not None:
        _out(lse, "lse", torch.float32, (b, h), di)
    st = _call(load_library().sink_attn_merge, di, stream,
               _ptr(partial_o), _ptr(partial_lse), b, s, h, d, _ptr(out), _ptr(lse))
    _check(st, "sink_attn_merge")
    return out, lse


def sink_attn_decode_shared(q, paged_k, paged_v, page_table, kv_lens, sinks, group_offsets, shared_pages,
                            max_shared_pages: int, sm_scale: float, splits=None, workspace=None, out=None,
                            lse=None, return_lse: bool = True, stream=None):
    """sink_attn_decode of a batch whose sequences share prompts: the pages that begin several
    sequences' page tables are read once for all of them.

    q [B, Hq, 64] bf16, paged_k/v [P, Hkv, 16, 64] bf16, page_table [B, max_pages] int32,
    kv_lens [B] int32 (whole sequences), sinks [Hq] fp32.  group_offsets [G + 1] int32: group g
    is sequences [group_offsets[g], group_offsets[g + 1]); shared_pages [G] int32: the pages that
    begin the page tables of all its sequences, at most max_shared_pages (best near the longest of them;
    the page table may be as wide as the model's context).
    splits: (shared, own) along the keys, default sink_attn_decode_shared_splits; (0, 1): every
    sequence reads all its pages for itself, in one launch.  workspace: (partial_o [B, shared + own,
    Hq, 64], partial_lse [B, shared + own, Hq]) fp32, allocated when not given, not used for (0, 1).  Returns (out [B, Hq, 64] bf16, lse [B, Hq] fp32 or None)."""
    b, hq, d = _shape(q, "q", 3)
    num_pages, hkv, page_size, kd = _shape(paged_k, "paged_k", 4)
    groups = _shape(shared_pages, "shared_pages", 1)[0]
    di = _inputs(("q", q, torch.bfloat16, (b, hq, d)), ("paged_k", paged_k, torch.bfloat16, (num_pages, hkv, page_size, d)),
                 ("paged_v", paged_v, torch.bfloat16, (num_pages, hkv, page_size, d)),
                 ("page_table", page_table, torch.int32, 2), ("kv_lens", kv_lens, torch.int32, (b,)),
                 ("sinks", sinks, torch.float32, (hq,)), ("group_offsets", group_offsets, torch.int32, (groups + 1,)),
                 ("shared_pages", shared_pages, torch.int32, (groups,)))
    if page_table.shape[0] != b:
        raise ValueError(f"page_table must have {b} rows, got {tuple(page_table.shape)}")
    max_pages, dev = page_table.shape[1], q.device
    most = _c_int(int(max_shared_pages), "max_shared_pages")
    if splits is None:
        splits = _shared_splits(b, groups, hq, hkv, most, max_pages, _sm_count(di))
    ss, so = (_c_int(int(v), "splits") for v in splits)
    if (ss, so) != (0, 1) and not (1 <= ss <= 255 and 1 <= so <= 256 - ss):  # no memory for what the call refuses
        raise ValueError(f"splits must be at least 1 each and at most 256 together, or (0, 1), got {(ss, so)}")
    scratch, rows, po, pl = None, b * (ss + so) * hq, 0, 0
    if ss == 0:
        pass  # every sequence by itself, in one launch
    elif workspace is None:
        if rows:
            scratch = _Scratch(4 * rows * (d + 1), di, stream)
            po, pl = scratch.ptr, scratch.ptr + 4 * rows * d
    else:
        po = _out(workspace[0], "workspace[0]", torch.float32, (b, ss + so, hq, d), di).data_ptr()
        pl = _out(workspace[1], "workspace[1]", torch.float32, (b, ss + so, hq), di).data_ptr()
    out = (_new((b, hq, d), torch.bfloat16, dev, stream) if out is None
           else _out(out, "out", torch.bfloat16, (b, hq, d), di))
    if lse is None and return_lse:
        lse = _new((b, hq), torch.float32, dev, stream)
    elif lse is not None:
        _out(lse, "lse", torch.float32, (b, hq), di)
    st = _call(load_library().sink_attn_decode_shared, di, stream, q.data_ptr(), paged_k.data_ptr(), paged_v.data_ptr(),
               page_table.data_ptr(), kv_lens.data_ptr(), sinks.data_ptr(), group_offsets.data_ptr(),
               shared_pages.data_ptr(), b, groups, hq, hkv, d, page_size, max_pages, num_pages, most, float(sm_scale),
               ss, so, po, pl, out.data_ptr(), _ptr(lse))
    del scratch
    _check(st, "sink_attn_decode_shared")
    return out, lse


_sms = {}


def _sm_count(di):
    """Multiprocessors of device ``di``."""
    if di not in _sms:
        _sms[di] = torch.cuda.get_device_properties(di).multi_processor_count
    return _sms[di]


def sink_attn_decode_shared_splits(batch: int, num_groups: int, num_qo_heads: int, num_kv_heads: int,
                                   max_shared_pages: int, max_pages: int, num_sms: int = 0):
    """(shared, own) split counts for sink_attn_decode_shared; num_sms 0: 152."""
    s, o = ctypes.c_int(), ctypes.c_int()
    load_library().sink_attn_decode_shared_splits(batch, num_groups, num_qo_heads, num_kv_heads, max_shared_pages,
                                                  max_pages, num_sms, ctypes.byref(s), ctypes.byref(o))
    return s.value, o.value


_shared_splits = functools.lru_cache(maxsize=4096)(sink_attn_decode_shared_splits)


def sink_attn_decode_splits(batch: int, num_kv_heads: int, max_kv_len: int, page_size: int = 16,
                            num_sms: int = 0) -> int:
    if num_sms <= 0 and torch.cuda.is_available():
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return load_library().sink_attn_decode_splits(batch, num_kv_heads, max_kv_len, page_size, num_sms)


def sink_attn_device_status(clear: bool = True) -> int:
    """Status word of the current device (synchronises); 0 when clean."""
    return load_library().sink_attn_device_status(int(bool(clear)))


def sink_attn_set_wait_timeout_ns(ns: int) -> None:
    load_library().sink_attn_set_wait_timeout_ns(int(ns))


def sink_attn_status_string(status: int) -> str:
    return load_library().sink_attn_status_string(int(status)).decode()


def sink_attn_abi_version() -> int:
    return load_library().sink_attn_abi_version()


def sink_attn_selftest_wait_timeout(timeout_ns: int = 1_000_000, stream=None) -> None:
    """Launch the bounded-wait diagnostic (records SA_ERR_TIMEOUT in the status word)."""
    di = torch.cuda.current_device() if stream is None else stream.device_index
    _check(_call(load_library().sink_attn_selftest_wait_timeout, di, stream, int(timeout_ns)),
           "sink_attn_selftest_wait_timeout")


# ----------------------------------------------------------------------------- around attention
def moe_router_topk_softmax(logits, top_k: int, topk_idx=None, topk_weight=None,
                            expert_counts=None, return_counts: bool = False, stream=None):
    """Top-K-then-softmax router over bf16 logits [T, E] (page "GPT-OSS on day 0",
    section "Kernels for GPT-OSS / MoE").  Returns (idx int32 [T, k], weight bf16
    [T, k]) and, with return_counts or a given expert_counts, the int32 [E] counts."""
    dev, di = _checked((("logits", logits, torch.bfloat16),))
    t, e = logits.shape
    k = int(top_k)
    topk_idx = (torch.empty((t, k), dtype=torch.int32, device=dev) if topk_idx is None
                else _out(topk_idx, "topk_idx", torch.int32, (t, k), di))
    topk_weight = (torch.empty((t, k), dtype=torch.bfloat16, device=dev) if topk_weight is None
                   else _out(topk_weight, "topk_weight", torch.bfloat16, (t, k), di))
    if expert_counts is None and return_counts:
        expert_counts = torch.empty((e,), dtype=torch.int32, device=dev)
    elif expert_counts is not None:
        _out(expert_counts, "expert_counts", torch.int32, (e,), di)
    st = _call(load_library().moe_router_topk_softmax, di, stream,
               _ptr(logits), t, e, k, _ptr(topk_idx), _ptr(topk_weight), _ptr(expert_counts))
    _check(st, "moe_router_topk_softmax")
    if expert_counts is not None:
        return topk_idx, topk_weight, expert_counts
    return topk_idx, topk_weight


def _rope_params(rope):
    r = dict(GPT_OSS_YARN if rope is None else rope)
    return (float(r["rope_base"]), float(r["factor"]), int(r["orig_len"]), float(r["beta_fast"]),
            float(r["beta_slow"]))


def _opt(named):
    """Validate the optional (name, tensor, dtype) triples that are not None."""
    for name, t, dt in named:
        if t is not None:
            _dev(t, name, dt)


def qkv_bias_rope(qkv, bias, cu_seqlens_q, num_qo_heads: int, num_kv_heads: int, kv_lens=None,
                  rope=None, q_out=None, k_out=None, v_out=None, stream=None):
    """QKV bias + YaRN rotation of q and k.  qkv bf16 [T, (Hq + 2 Hkv) * 64] -> (q [T, Hq, 64],
    k [T, Hkv, 64], v [T, Hkv, 64]) bf16.  rope: dict like GPT_OSS_YARN (default)."""
    dev, di = _checked((("qkv", qkv, torch.bfloat16), ("cu_seqlens_q", cu_seqlens_q, torch.int32)))
    _opt((("bias", bias, torch.bfloat16), ("kv_lens", kv_lens, torch.int32)))
    t = qkv.shape[0]
    hq, hkv, d = int(num_qo_heads), int(num_kv_heads), 64
    _same_device(di, ("bias", bias), ("cu_seqlens_q", cu_seqlens_q), ("kv_lens", kv_lens))
    q_out = torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev) if q_out is None else q_out
    k_out = torch.empty((t, hkv, d), dtype=torch.bfloat16, device=dev) if k_out is None else k_out
    v_out = torch.empty((t, hkv, d), dtype=torch.bfloat16, device=dev) if v_out is None else v_out
    for name, x, h in (("q_out", q_out, hq), ("k_out", k_out, hkv), ("v_out", v_out, hkv)):
        _out(x, name, torch.bfloat16, (t, h, d), di)
    st = _call(load_library().qkv_bias_rope, di, stream,
               _ptr(qkv), _ptr(bias), _ptr(cu_seqlens_q), _ptr(kv_lens), cu_seqlens_q.numel() - 1, t, hq, hkv,
               qkv.shape[1] // (hq + 2 * hkv), *_rope_params(rope), _ptr(q_out), _ptr(k_out), _ptr(v_out))
    _check(st, "qkv_bias_rope")
    return q_out, k_out, v_out


def qkv_bias_rope_append_paged(qkv, bias, cu_seqlens_q, kv_lens, paged_k, paged_v, page_table,
                               num_qo_heads: int, rope=None, q_out=None, stream=None):
    """QKV bias + YaRN rotation; q returned [T, Hq, 64], k and v written in place into the
    paged cache [num_pages, Hkv, 16, 64] at each new token's position."""
    dev, di = _checked((("qkv", qkv, torch.bfloat16), ("cu_seqlens_q", cu_seqlens_q, torch.int32),
                        ("kv_lens", kv_lens, torch.int32), ("paged_k", paged_k, torch.bfloat16),
                        ("paged_v", paged_v, torch.bfloat16), ("page_table", page_table, torch.int32)))
    _opt((("bias", bias, torch.bfloat16),))
    t = qkv.shape[0]
    num_pages, hkv, page_size, d = paged_k.shape
    hq = int(num_qo_heads)
    _same_device(di, ("bias", bias), ("cu_seqlens_q", cu_seqlens_q), ("kv_lens", kv_lens),
                 ("paged_k", paged_k), ("paged_v", paged_v), ("page_table", page_table))
    q_out = torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev) if q_out is None else q_out
    _out(q_out, "q_out", torch.bfloat16, (t, hq, d), di)
    st = _call(load_library().qkv_bias_rope_append_paged, di, stream,
               _ptr(qkv), _ptr(bias), _ptr(cu_seqlens_q), _ptr(kv_lens), cu_seqlens_q.numel() - 1, t, hq, hkv,
               qkv.shape[1] // (hq + 2 * hkv), *_rope_params(rope), _ptr(q_out), _ptr(paged_k), _ptr(paged_v),
               _ptr(page_table), page_size, page_table.shape[1], num_pages)
    _check(st, "qkv_bias_rope_append_paged")
    return q_out


def linear_bias(x, w, bias=None, out=None, stream=None):
    """out [M, N] = x [M, K] @ w[N, K]^T + bias[N] on the tcgen05 tensor cores, bf16 in and out,
    the fp32 accumulator seeded with the bias (page "GPT-OSS on day 0", section "Kernels for
    GPT-OSS / MoE")."""
    dev, di = _checked((("x", x, torch.bfloat16), ("w", w, torch.bfloat16)))
    _opt((("bias", bias, torch.bfloat16),))
    m, k = x.shape
    n = w.shape[0]
    if w.shape[1] != k:
        raise ValueError(f"w is {tuple(w.shape)}, expected [N, {k}]")
    _same_device(di, ("w", w), ("bias", bias))
    out = torch.empty((m, n), dtype=torch.bfloat16, device=dev) if out is None else out
    _out(out, "out", torch.bfloat16, (m, n), di)
    st = _call(load_library().linear_bias, di, stream, _ptr(x), _ptr(w), _ptr(bias), m, n, k, _ptr(out))
    _check(st, "linear_bias")
    return out


def lora_workspace_bytes(m: int, k: int, rank: int) -> int:
    """Bytes of workspace for lora_linear_bias of m tokens."""
    n = ctypes.c_longlong()
    load_library().lora_workspace_bytes(_c_int(m, "m"), _c_int(k, "k"), _c_int(rank, "rank"), ctypes.byref(n))
    return n.value


_lora_bytes = functools.lru_cache(maxsize=4096)(lora_workspace_bytes)


def lora_linear_bias(x, w, lora_a, lora_b, adapter_idx, bias=None, lora_scale=None, out=None, workspace=None,
                     stream=None):
    """linear_bias with the low-rank adapters of many requests at once beside it:
    out[m] = x[m] @ w^T + bias + lora_scale[a] * (x[m] @ lora_a[a]^T) @ lora_b[a]^T for
    a = adapter_idx[m], without the last term where adapter_idx[m] is negative.

    x [M, K] bf16, w [N, K] bf16, lora_a [L, R, K] bf16, lora_b [L, N, R] bf16 (R a multiple of 8,
    at most 128; L at most 1024), adapter_idx [M] int32, bias [N] bf16 or None, lora_scale [L]
    fp32 or None (1).  workspace: a uint8 tensor of at least lora_workspace_bytes(M, K, R) bytes,
    allocated when not given.  Returns out [M, N] bf16."""
    n, k = _shape(w, "w", 2)
    l, r, _ = _shape(lora_a, "lora_a", 3)
    m = _shape(x, "x", 2)[0]
    named = [("x", x, torch.bfloat16, (m, k)), ("w", w, torch.bfloat16, (n, k)), ("lora_a", lora_a, torch.bfloat16, (l, r, k)),
             ("lora_b", lora_b, torch.bfloat16, (l, n, r)), ("adapter_idx", adapter_idx, torch.int32, (m,))]
    if bias is not None:
        named.append(("bias", bias, torch.bfloat16, (n,)))
    if lora_scale is not None:
        named.append(("lora_scale", lora_scale, torch.float32, (l,)))
    di = _inputs(*named)
    lib = load_library()
    need, scratch, ws = _lora_bytes(m, k, r), None, 0
    if workspace is None:
        if need:
            scratch = _Scratch(need, di, stream)
            ws = scratch.ptr
    else:
        _dev(workspace, "workspace", torch.uint8)
        _same_device(di, ("workspace", workspace))
        if workspace.numel() < need:
            raise ValueError(f"workspace must have at least {need} bytes, got {workspace.numel()}")
        ws = workspace.data_ptr()
    out = _product_output(out, m, n, x, di, stream)
    st = _call(lib.lora_linear_bias, di, stream, x.data_ptr(), w.data_ptr(), _ptr(bias), lora_a.data_ptr(),
               lora_b.data_ptr(), _ptr(lora_scale), adapter_idx.data_ptr(), m, n, k, r, l, ws, out.data_ptr())
    del scratch
    _check(st, "lora_linear_bias")
    return out


def moe_router(x, w_router, bias, top_k: int, topk_idx=None, topk_weight=None, expert_counts=None,
               return_counts: bool = False, stream=None):
    """Router projection + bias + bf16 logits + Top-K softmax in one tcgen05 kernel:
    x [T, hidden] bf16, w_router [E, hidden] bf16, bias [E] bf16 or None.  Returns
    (idx int32 [T, k], weight bf16 [T, k]) and the int32 [E] counts when asked."""
    dev, di = _checked((("x", x, torch.bfloat16), ("w_router", w_router, torch.bfloat16)))
    _opt((("bias", bias, torch.bfloat16),))
    t, hidden = x.shape
    e = w_router.shape[0]
    if w_router.shape[1] != hidden:
        raise ValueError(f"w_router is {tuple(w_router.shape)}, expected [E, {hidden}]")
    k = int(top_k)
    _same_device(di, ("w_router", w_router), ("bias", bias))
    topk_idx = (torch.empty((t, k), dtype=torch.int32, device=dev) if topk_idx is None
                else _out(topk_idx, "topk_idx", torch.int32, (t, k), di))
    topk_weight = (torch.empty((t, k), dtype=torch.bfloat16, device=dev) if topk_weight is None
                   else _out(topk_weight, "topk_weight", torch.bfloat16, (t, k), di))
    if expert_counts is None and return_counts:
        expert_counts = torch.empty((e,), dtype=torch.int32, device=dev)
    elif expert_counts is not None:
        _out(expert_counts, "expert_counts", torch.int32, (e,), di)
    st = _call(load_library().moe_router, di, stream, _ptr(x), _ptr(w_router), _ptr(bias), t, hidden, e, k,
               _ptr(topk_idx), _ptr(topk_weight), _ptr(expert_counts))
    _check(st, "moe_router")
    if expert_counts is not None:
        return topk_idx, topk_weight, expert_counts
    return topk_idx, topk_weight


def moe_router_scores(logits, top_k: int, score: str = "softmax", bias=None, num_groups: int = 1, top_groups: int = 1,
                      renormalize: bool = True, scale: float = 1.0, topk_idx=None, topk_weight=None,
                      expert_counts=None, return_counts: bool = False, stream=None):
    """Router by scores: s = softmax or sigmoid of the logits [T, E] (bf16 or fp32) over all experts,
    the top_k largest s + bias among the top_groups best of num_groups groups of consecutive
    experts (a group's merit: the sum of its two largest s + bias), largest first, equal values in
    favour of the lower index; weights scale * s, divided by the sum of the chosen s with
    renormalize.  bias [E] fp32 or None.  Returns (idx int32 [T, k], weight bf16 [T, k]) and the
    int32 [E] counts when asked."""
    if score not in ("softmax", "sigmoid"):
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    fp32 = isinstance(logits, torch.Tensor) and logits.dtype is torch.float32
    t, e = _shape(logits, "logits", 2)
    named = [("logits", logits, torch.float32 if fp32 else torch.bfloat16, (t, e))]
    if bias is not None:
        named.append(("bias", bias, torch.float32, (e,)))
    di, dev = _inputs(*named), logits.device
    k = _c_int(int(top_k), "top_k")
    if not 1 <= k <= 8:  # no memory for what the call refuses
        raise ValueError(f"top_k must be 1 to 8, got {k}")
    topk_idx = (_new((t, k), torch.int32, dev, stream) if topk_idx is None
                else _out(topk_idx, "topk_idx", torch.int32, (t, k), di))
    topk_weight = (_new((t, k), torch.bfloat16, dev, stream) if topk_weight is None
                   else _out(topk_weight, "topk_weight", torch.bfloat16, (t, k), di))
    if expert_counts is None and return_counts:
        expert_counts = _new((e,), torch.int32, dev, stream)
    elif expert_counts is not None:
        _out(expert_counts, "expert_counts", torch.int32, (e,), di)
    st = _call(load_library().moe_router_scores, di, stream, logits.data_ptr(), int(fp32), t, e, k,
               int(score == "sigmoid"), _ptr(bias), _c_int(int(num_groups), "num_groups"),
               _c_int(int(top_groups), "top_groups"), int(bool(renormalize)), float(scale), topk_idx.data_ptr(),
               topk_weight.data_ptr(), _ptr(expert_counts))
    _check(st, "moe_router_scores")
    if expert_counts is not None:
        return topk_idx, topk_weight, expert_counts
    return topk_idx, topk_weight


# ----------------------------------------------------------------------------- the expert layer
# SwiGLU constants of the public GPT-OSS model configuration (the pages name
# SwiGLU but give no constants).
GPT_OSS_SWIGLU = dict(alpha=1.702, limit=7.0)


_C_INT = 2 ** 31 - 1
_MAX_EXPERTS = 256  # of moe_experts.h


def _c_int(v, name):
    """v, which has to survive the passage through a C int."""
    if not -_C_INT <= v <= _C_INT:
        raise ValueError(f"{name} is {v}, beyond 32 bits")
    return v


def _new(shape, dtype, dev, stream):
    """An output, from the memory of the stream that will write it: the current stream's may
    still be in use there, or be given out there again while the kernel runs."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


class _Scratch:
    """Memory of a call's own, from the memory of the stream that uses it: given back when the call
    has been enqueued, so that whatever the stream does next may have it (a third of what a tensor
    costs the host)."""
    __slots__ = ("ptr",)

    def __init__(self, nbytes, di, stream):
        s = torch._C._cuda_getCurrentRawStream(di) if stream is None else stream.cuda_stream
        if torch._C._cuda_getDevice() == di:
            self.ptr = torch._C._cuda_cudaCachingAllocator_raw_alloc(nbytes, s)
        else:
            with torch.cuda.device(di):
                self.ptr = torch._C._cuda_cudaCachingAllocator_raw_alloc(nbytes, s)

    def __del__(self):
        if getattr(self, "ptr", 0):
            torch._C._cuda_cudaCachingAllocator_raw_delete(self.ptr)


def _inputs(*named):
    """Validate (name, tensor, dtype, shape) tuples: CUDA, dtype, contiguous, shape (an int: any
    shape of that many dimensions), all on the first tensor's device.  Returns that device's
    index.  Optional tensors are left out by the caller when they are None."""
    di = -1
    for name, t, dt, shape in named:
        try:  # what a good call's tensors but the first are
            if t.dtype is dt and t.shape == shape and t.get_device() == di >= 0 and t.is_contiguous() and t.numel() <= _C_INT:
                continue
        except AttributeError:
            pass
        if not isinstance(t, torch.Tensor) or t.dtype is not dt or not t.is_contiguous():
            _dev(t, name, dt)  # raises
        d = t.get_device()  # -1 on the CPU
        if d != di:
            if di >= 0:
                _same_device(di, (name, t))  # raises
            di = d
        if d < 0:
            _dev(t, name, dt)  # raises
        if t.numel() > _C_INT:
            for v in t.shape:
                _c_int(v, f"a dimension of {name}")
        if t.shape != shape and t.dim() != shape:
            want = f"of {shape} dimensions" if isinstance(shape, int) else list(shape)
            raise ValueError(f"{name} must be {want}, got {tuple(t.shape)}")
    return di


def _shape(t, name, dims):
    """The shape of something that may not be a tensor of ``dims`` dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must be of {dims} dimensions, got {tuple(t.shape)}")
    return t.shape


def moe_group_rows(topk_idx, num_experts: int, expert_offsets=None, row_token=None, pair_row=None,
                   stream=None):
    """Sort the (token, expert) pairs of topk_idx [T, k] int32 by expert, stably.

    Returns (expert_offsets int32 [E + 1], row_token int32 [T * k], pair_row int32 [T, k]):
    expert e owns rows [expert_offsets[e], expert_offsets[e + 1]), row r reads token
    row_token[r], and pair (t, i) is row pair_row[t, i].  A negative index is a pair without
    expert (pair_row -1); row_token is -1 behind the last row."""
    di = _inputs(("topk_idx", topk_idx, torch.int32, 2))
    t, k = topk_idx.shape
    e = _c_int(int(num_experts), "num_experts")
    dev = topk_idx.device
    # no memory for a number of experts that the call refuses
    expert_offsets = (_new(min(max(e, 0), _MAX_EXPERTS) + 1, torch.int32, dev, stream) if expert_offsets is None
                      else _out(expert_offsets, "expert_offsets", torch.int32, (e + 1,), di))
    row_token = (_new(t * k, torch.int32, dev, stream) if row_token is None
                 else _out(row_token, "row_token", torch.int32, (t * k,), di))
    pair_row = (_new((t, k), torch.int32, dev, stream) if pair_row is None
                else _out(pair_row, "pair_row", torch.int32, (t, k), di))
    st = _call(load_library().moe_group_rows, di, stream, topk_idx.data_ptr(), t, k, e, expert_offsets.data_ptr(),
               row_token.data_ptr(), pair_row.data_ptr())
    _check(st, "moe_group_rows")
    return expert_offsets, row_token, pair_row


def moe_combine(y, pair_row, topk_weight, out=None, stream=None):
    """out[t] = sum_i topk_weight[t, i] * y[pair_row[t, i]]: y [R, H] bf16, pair_row [T, k]
    int32 (-1 adds nothing), topk_weight [T, k] bf16.  Returns out [T, H] bf16."""
    t, k = _shape(pair_row, "pair_row", 2)
    di = _inputs(("y", y, torch.bfloat16, 2), ("pair_row", pair_row, torch.int32, (t, k)),
                 ("topk_weight", topk_weight, torch.bfloat16, (t, k)))
    r, h = y.shape
    out = (_new((t, h), torch.bfloat16, y.device, stream) if out is None
           else _out(out, "out", torch.bfloat16, (t, h), di))
    st = _call(load_library().moe_combine, di, stream, y.data_ptr(), pair_row.data_ptr(), topk_weight.data_ptr(), r,
               t, k, h, out.data_ptr())
    _check(st, "moe_combine")
    return out


def _product_output(out, rows, n, x, di, stream):
    return (_new((rows, n), torch.bfloat16, x.device, stream) if out is None
            else _out(out, "out", torch.bfloat16, (rows, n), di))


def _grouped(where, x, w, expert_offsets, bias, row_token, out, stream, act=()):
    """The grouped products on bf16 operands; act: SwiGLU's (alpha, limit) or ()."""
    e, n, k = _shape(w, "w", 3)
    x_rows = _shape(x, "x", 2)[0]
    named = [("x", x, torch.bfloat16, (x_rows, k)), ("w", w, torch.bfloat16, (e, n, k)),
             ("expert_offsets", expert_offsets, torch.int32, (e + 1,))]
    if bias is not None:
        named.append(("bias", bias, torch.bfloat16, (e, n)))
    if row_token is not None:
        named.append(("row_token", row_token, torch.int32, 1))
    di = _inputs(*named)
    rows = x_rows if row_token is None else row_token.shape[0]
    out = _product_output(out, rows, n // 2 if act else n, x, di, stream)
    st = _call(getattr(load_library(), where), di, stream, x.data_ptr(), w.data_ptr(), _ptr(bias),
               expert_offsets.data_ptr(), _ptr(row_token), x_rows, rows, e, n, k, *act, out.data_ptr())
    _check(st, where)
    return out


def grouped_linear_bias(x, w, expert_offsets, bias=None, row_token=None, out=None, stream=None):
    """One linear layer per expert on its ragged group of rows, on the tcgen05 tensor cores.

    x [X, K] bf16, w [E, N, K] bf16, expert_offsets [E + 1] int32, bias [E, N] bf16 or None;
    row r of expert e gives out[r] = x[row_token[r]] @ w[e]^T + bias[e] (row_token None: x[r]).
    Returns out [R, N] bf16; rows outside every group are left as they were (uninitialised
    when ``out`` is not given)."""
    return _grouped("grouped_linear_bias", x, w, expert_offsets, bias, row_token, out, stream)


def grouped_linear_swiglu(x, w, expert_offsets, bias=None, row_token=None,
                          alpha: float = GPT_OSS_SWIGLU["alpha"], limit: float = GPT_OSS_SWIGLU["limit"],
                          out=None, stream=None):
    """grouped_linear_bias followed by the clamped SwiGLU on interleaved gate (even) and up
    (odd) features, before the one rounding to bf16: g * sigmoid(alpha g) * (u + 1) with
    g = min(gate, limit), u = clamp(up, -limit, limit).  Returns out [R, N / 2] bf16."""
    return _grouped("grouped_linear_swiglu", x, w, expert_offsets, bias, row_token, out, stream,
                    (float(alpha), float(limit)))


# ----------------------------------------------------------------------------- MXFP4
def mxfp4_scale_columns(k: int) -> int:
    """Scale bytes per row of a K-wide MXFP4 matrix: K / 32 rounded up to a multiple of 16."""
    return (int(k) // 32 + 15) // 16 * 16


def mxfp4_quantize(x, codes=None, scales=None, stream=None):
    """Quantise x [..., K] (bf16 or fp32, K a multiple of 32) to MXFP4: blocks of 32 values
    share the scale 2^(floor(log2 max|x|) - 2), values round to the nearest E2M1 (ties to
    even, at most 6).  Returns (codes uint8 [..., K / 2], scales uint8
    [..., mxfp4_scale_columns(K)])."""
    fp32 = isinstance(x, torch.Tensor) and x.dtype is torch.float32
    _dev(x, "x", torch.float32 if fp32 else torch.bfloat16)
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    di, dev, lead, k = x.get_device(), x.device, x.shape[:-1], _c_int(x.shape[-1], "K")
    codes = (_new((*lead, k // 2), torch.uint8, dev, stream) if codes is None
             else _out(codes, "codes", torch.uint8, (*lead, k // 2), di))
    s = mxfp4_scale_columns(k)
    scales = (_new((*lead, s), torch.uint8, dev, stream) if scales is None
              else _out(scales, "scales", torch.uint8, (*lead, s), di))
    st = _call(load_library().mxfp4_quantize, di, stream, x.data_ptr(), int(fp32), lead.numel(), k,
               codes.data_ptr(), scales.data_ptr())
    _check(st, "mxfp4_quantize")
    return codes, scales


def mxfp4_dequantize(codes, scales, out=None, stream=None):
    """The bf16 values [..., K] of MXFP4 codes [..., K / 2] and scales (as mxfp4_quantize
    returns them)."""
    _dev(codes, "codes", torch.uint8)
    if codes.dim() < 1:
        raise ValueError("codes must have at least one dimension")
    # as mxfp4_quantize: K passes through a C int, the number of rows does not
    di, k, lead = codes.get_device(), _c_int(2 * codes.shape[-1], "K"), codes.shape[:-1]
    _out(scales, "scales", torch.uint8, (*lead, mxfp4_scale_columns(k)), di)
    out = (_new((*lead, k), torch.bfloat16, codes.device, stream) if out is None
           else _out(out, "out", torch.bfloat16, (*lead, k), di))
    st = _call(load_library().mxfp4_dequantize, di, stream, codes.data_ptr(), scales.data_ptr(), lead.numel(), k,
               out.data_ptr())
    _check(st, "mxfp4_dequantize")
    return out


def mxfp4_linear_bias(x_codes, x_scales, w_codes, w_scales, bias=None, out=None, stream=None):
    """linear_bias with both operands in MXFP4 (block-scaled tcgen05 products): x [M, K] and
    w [N, K] as codes [., K / 2] and scales, bias [N] bf16 or None.  Returns [M, N] bf16."""
    m, half = _shape(x_codes, "x_codes", 2)
    n = _shape(w_codes, "w_codes", 2)[0]
    s = mxfp4_scale_columns(2 * half)
    named = [("x_codes", x_codes, torch.uint8, (m, half)), ("x_scales", x_scales, torch.uint8, (m, s)),
             ("w_codes", w_codes, torch.uint8, (n, half)), ("w_scales", w_scales, torch.uint8, (n, s))]
    if bias is not None:
        named.append(("bias", bias, torch.bfloat16, (n,)))
    di = _inputs(*named)
    out = _product_output(out, m, n, x_codes, di, stream)
    st = _call(load_library().mxfp4_linear_bias, di, stream, x_codes.data_ptr(), x_scales.data_ptr(),
               w_codes.data_ptr(), w_scales.data_ptr(), _ptr(bias), m, n, 2 * half, out.data_ptr())
    _check(st, "mxfp4_linear_bias")
    return out


def _grouped_mxfp4(where, x_codes, x_scales, w_codes, w_scales, expert_offsets, bias, row_token, out, stream, act=()):
    """The grouped products on MXFP4 operands; act: SwiGLU's (alpha, limit) or ()."""
    e, n, half = _shape(w_codes, "w_codes", 3)
    x_rows, s = _shape(x_codes, "x_codes", 2)[0], mxfp4_scale_columns(2 * half)
    named = [("x_codes", x_codes, torch.uint8, (x_rows, half)), ("x_scales", x_scales, torch.uint8, (x_rows, s)),
             ("w_codes", w_codes, torch.uint8, (e, n, half)), ("w_scales", w_scales, torch.uint8, (e, n, s)),
             ("expert_offsets", expert_offsets, torch.int32, (e + 1,))]
    if bias is not None:
        named.append(("bias", bias, torch.bfloat16, (e, n)))
    if row_token is not None:
        named.append(("row_token", row_token, torch.int32, 1))
    di = _inputs(*named)
    rows = x_rows if row_token is None else row_token.shape[0]
    out = _product_output(out, rows, n // 2 if act else n, x_codes, di, stream)
    st = _call(getattr(load_library(), where), di, stream, x_codes.data_ptr(), x_scales.data_ptr(),
               w_codes.data_ptr(), w_scales.data_ptr(), _ptr(bias), expert_offsets.data_ptr(), _ptr(row_token),
               x_rows, rows, e, n, 2 * half, *act, out.data_ptr())
    _check(st, where)
    return out


def grouped_mxfp4_linear_bias(x_codes, x_scales, w_codes, w_scales, expert_offsets, bias=None, row_token=None,
                              out=None, stream=None):
    """grouped_linear_bias with both operands in MXFP4: x [X, K] and w [E, N, K] as codes
    [., K / 2] and scales (row_token gathers rows of both)."""
    return _grouped_mxfp4("grouped_mxfp4_linear_bias", x_codes, x_scales, w_codes, w_scales, expert_offsets, bias,
                          row_token, out, stream)


def grouped_mxfp4_linear_swiglu(x_codes, x_scales, w_codes, w_scales, expert_offsets, bias=None, row_token=None,
                                alpha: float = GPT_OSS_SWIGLU["alpha"], limit: float = GPT_OSS_SWIGLU["limit"],
                                out=None, stream=None):
    """grouped_linear_swiglu with both operands in MXFP4."""
    return _grouped_mxfp4("grouped_mxfp4_linear_swiglu", x_codes, x_scales, w_codes, w_scales, expert_offsets, bias,
                          row_token, out, stream, (float(alpha), float(limit)))


# ----------------------------------------------------------------------------- q rotated on chip
def qkv_bias_rope_kv(qkv, bias, cu_seqlens_q, num_qo_heads: int, num_kv_heads: int, kv_lens=None,
                     rope=None, k_out=None, v_out=None, rope_table=None, stream=None):
    """K/V half of qkv_bias_rope for the *_qkv attention calls: k (biased, rotated) and v
    (biased) written contiguous [T, Hkv, 64] bf16, plus the per-token (cos, sin) table
    [T, 32, 2] fp32 those calls apply to q.  Returns (k, v, rope_table)."""
    dev, di = _checked((("qkv", qkv, torch.bfloat16), ("cu_seqlens_q", cu_seqlens_q, torch.int32)))
    _opt((("bias", bias, torch.bfloat16), ("kv_lens", kv_lens, torch.int32)))
    t = qkv.shape[0]
    hq, hkv, d = int(num_qo_heads), int(num_kv_heads), 64
    _same_device(di, ("bias", bias), ("cu_seqlens_q", cu_seqlens_q), ("kv_lens", kv_lens))
    k_out = torch.empty((t, hkv, d), dtype=torch.bfloat16, device=dev) if k_out is None else k_out
    v_out = torch.empty((t, hkv, d), dtype=torch.bfloat16, device=dev) if v_out is None else v_out
    rope_table = (torch.empty((t, d // 2, 2), dtype=torch.float32, device=dev) if rope_table is None
                  else rope_table)
    _out(k_out, "k_out", torch.bfloat16, (t, hkv, d), di)
    _out(v_out, "v_out", torch.bfloat16, (t, hkv, d), di)
    _out(rope_table, "rope_table", torch.float32, (t, d // 2, 2), di)
    st = _call(load_library().qkv_bias_rope_kv, di, stream,
               _ptr(qkv), _ptr(bias), _ptr(cu_seqlens_q), _ptr(kv_lens), cu_seqlens_q.numel() - 1, t, hq, hkv,
               qkv.shape[1] // (hq + 2 * hkv), *_rope_params(rope), _ptr(k_out), _ptr(v_out), _ptr(rope_table))
    _check(st, "qkv_bias_rope_kv")
    return k_out, v_out, rope_table


def qkv_bias_rope_append_paged_kv(qkv, bias, cu_seqlens_q, kv_lens, paged_k, paged_v, page_table,
                                  num_qo_heads: int, rope=None, rope_table=None, stream=None):
    """K/V half of qkv_bias_rope_append_paged: k and v written in place into the paged
    cache at each new token's position, and the (cos, sin) table [T, 32, 2] fp32 of the
    new tokens returned for the *_qkv attention calls."""
    dev, di = _checked((("qkv", qkv, torch.bfloat16), ("cu_seqlens_q", cu_seqlens_q, torch.int32),
                        ("kv_lens", kv_lens, torch.int32), ("paged_k", paged_k, torch.bfloat16),
                        ("paged_v", paged_v, torch.bfloat16), ("page_table", page_table, torch.int32)))
    _opt((("bias", bias, torch.bfloat16),))
    t = qkv.shape[0]
    num_pages, hkv, page_size, d = paged_k.shape
    hq = int(num_qo_heads)
    _same_device(di, ("bias", bias), ("cu_seqlens_q", cu_seqlens_q), ("kv_lens", kv_lens),
                 ("paged_k", paged_k), ("paged_v", paged_v), ("page_table", page_table))
    rope_table = (torch.empty((t, d // 2, 2), dtype=torch.float32, device=dev) if rope_table is None
                  else rope_table)
    _out(rope_table, "rope_table", torch.float32, (t, d // 2, 2), di)
    st = _call(load_library().qkv_bias_rope_append_paged_kv, di, stream,
               _ptr(qkv), _ptr(bias), _ptr(cu_seqlens_q), _ptr(kv_lens), cu_seqlens_q.numel() - 1, t, hq, hkv,
               qkv.shape[1] // (hq + 2 * hkv), *_rope_params(rope), _ptr(paged_k), _ptr(paged_v),
               _ptr(page_table), page_size, page_table.shape[1], num_pages, _ptr(rope_table))
    _check(st, "qkv_bias_rope_append_paged_kv")
    return rope_table


def sink_attn_prefill_qkv(qkv, qkv_bias, rope_table, k, v, sinks, cu_seqlens, max_seqlen: int,
                          sm_scale: float, num_qo_heads: int, causal: bool = True, out=None, lse=None,
                          return_lse: bool = True, stream=None):
    """sink_attn_prefill with q taken from the projection output qkv [T, (Hq + 2 Hkv) * 64]:
    the query bias and the rotation by rope_table (from qkv_bias_rope_kv) are applied on
    chip; k, v as written by qkv_bias_rope_kv."""
    dev, di = _checked((("qkv", qkv, torch.bfloat16), ("rope_table", rope_table, torch.float32),
                        ("k", k, torch.bfloat16), ("v", v, torch.bfloat16), ("sinks", sinks, torch.float32),
                        ("cu_seqlens", cu_seqlens, torch.int32)))
    _opt((("qkv_bias", qkv_bias, torch.bfloat16),))
    t = qkv.shape[0]
    hq = int(num_qo_heads)
    _, hkv, d = k.shape
    if k.shape != (t, hkv, d) or v.shape != k.shape or qkv.shape[1] != (hq + 2 * hkv) * d:
        raise ValueError("qkv must be [T, (Hq + 2 Hkv) * D] and k, v [T, Hkv, D]")
    if tuple(rope_table.shape) != (t, d // 2, 2):
        raise ValueError(f"rope_table must be {(t, d // 2, 2)}")
    _same_device(di, ("qkv_bias", qkv_bias), ("rope_table", rope_table), ("k", k), ("v", v), ("sinks", sinks),
                 ("cu_seqlens", cu_seqlens))
    out = (torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev) if out is None
           else _out(out, "out", torch.bfloat16, (t, hq, d), di))
    if lse is None and return_lse:
        lse = torch.empty((t, hq), dtype=torch.float32, device=dev)
    elif lse is not None:
        _out(lse, "lse", torch.float32, (t, hq), di)
    st = _call(load_library().sink_attn_prefill_qkv, di, stream,
               _ptr(qkv), _ptr(qkv_bias), _ptr(rope_table), _ptr(k), _ptr(v), _ptr(sinks), _ptr(cu_seqlens),
               cu_seqlens.numel() - 1, t, int(max_seqlen), hq, hkv, d, float(sm_scale), int(bool(causal)),
               _ptr(out), _ptr(lse))
    _check(st, "sink_attn_prefill_qkv")
    return out, lse


def sink_attn_prefill_paged_qkv(qkv, qkv_bias, rope_table, paged_k, paged_v, page_table, cu_seqlens_q,
                                kv_lens, sinks, max_q_len: int, sm_scale: float, num_qo_heads: int,
                                causal: bool = True, out=None, lse=None, return_lse: bool = True,
                                stream=None):
    """sink_attn_prefill_paged with q taken from the projection output (see
    sink_attn_prefill_qkv); the paged cache and rope_table as written by
    qkv_bias_rope_append_paged_kv."""
    dev, di = _checked((("qkv", qkv, torch.bfloat16), ("rope_table", rope_table, torch.float32),
                        ("paged_k", paged_k, torch.bfloat16), ("paged_v", paged_v, torch.bfloat16),
                        ("page_table", page_table, torch.int32), ("cu_seqlens_q", cu_seqlens_q, torch.int32),
                        ("kv_lens", kv_lens, torch.int32), ("sinks", sinks, torch.float32)))
    _opt((("qkv_bias", qkv_bias, torch.bfloat16),))
    t = qkv.shape[0]
    hq = int(num_qo_heads)
    num_pages, hkv, page_size, d = paged_k.shape
    if qkv.shape[1] != (hq + 2 * hkv) * d or tuple(rope_table.shape) != (t, d // 2, 2):
        raise ValueError("qkv must be [T, (Hq + 2 Hkv) * D] and rope_table [T, D / 2, 2]")
    _same_device(di, ("qkv_bias", qkv_bias), ("rope_table", rope_table), ("paged_k", paged_k),
                 ("paged_v", paged_v), ("page_table", page_table), ("cu_seqlens_q", cu_seqlens_q),
                 ("kv_lens", kv_lens), ("sinks", sinks))
    out = (torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev) if out is None
           else _out(out, "out", torch.bfloat16, (t, hq, d), di))
    if lse is None and return_lse:
        lse = torch.empty((t, hq), dtype=torch.float32, device=dev)
    elif lse is not None:
        _out(lse, "lse", torch.float32, (t, hq), di)
    st = _call(load_library().sink_attn_prefill_paged_qkv, di, stream,
               _ptr(qkv), _ptr(qkv_bias), _ptr(rope_table), _ptr(paged_k), _ptr(paged_v), _ptr(page_table),
               _ptr(cu_seqlens_q), _ptr(kv_lens), _ptr(sinks), cu_seqlens_q.numel() - 1, t, int(max_q_len), hq,
               hkv, d, page_size, page_table.shape[1], num_pages, float(sm_scale), int(bool(causal)), _ptr(out),
               _ptr(lse))
    _check(st, "sink_attn_prefill_paged_qkv")
    return out, lse


def sink_attn_decode_qkv(qkv, qkv_bias, rope_table, paged_k, paged_v, page_table, kv_lens, sinks,
                         sm_scale: float, num_qo_heads: int, num_splits: int = 1, out=None, lse=None,
                         return_lse: bool = True, stream=None):
    """sink_attn_decode with q taken from the projection output qkv [B, (Hq + 2 Hkv) * 64] (one
    new token per sequence): bias and rotation by row b of rope_table [B, 32, 2] applied in
    the kernel.  num_splits > 1 returns the fp32 partials, as sink_attn_decode does."""
    dev, di = _checked((("qkv", qkv, torch.bfloat16), ("rope_table", rope_table, torch.float32),
                        ("paged_k", paged_k, torch.bfloat16), ("paged_v", paged_v, torch.bfloat16),
                        ("page_table", page_table, torch.int32), ("kv_lens", kv_lens, torch.int32),
                        ("sinks", sinks, torch.float32)))
    _opt((("qkv_bias", qkv_bias, torch.bfloat16),))
    b = qkv.shape[0]
    hq = int(num_qo_heads)
    num_pages, hkv, page_size, d = paged_k.shape
    if qkv.shape[1] != (hq + 2 * hkv) * d or tuple(rope_table.shape) != (b, d // 2, 2):
        raise ValueError("qkv must be [B, (Hq + 2 Hkv) * D] and rope_table [B, D / 2, 2]")
    _same_device(di, ("qkv_bias", qkv_bias), ("rope_table", rope_table), ("paged_k", paged_k),
                 ("paged_v", paged_v), ("page_table", page_table), ("kv_lens", kv_lens), ("sinks", sinks))
    s = int(num_splits)
    out, lse = _decode_outputs(out, lse, return_lse, b, s, hq, d, dev, di)
    st = _call(load_library().sink_attn_decode_qkv, di, stream,
               _ptr(qkv), _ptr(qkv_bias), _ptr(rope_table), _ptr(paged_k), _ptr(paged_v), _ptr(page_table),
               _ptr(kv_lens), _ptr(sinks), b, hq, hkv, d, page_size, page_table.shape[1], num_pages,
               float(sm_scale), s, _ptr(out), _ptr(lse))
    _check(st, "sink_attn_decode_qkv")
    return out, lse
