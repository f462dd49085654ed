"""The expert layer's C ABI and its Python wrappers on the CPU: bad arguments are refused with a
status code (or an exception) before anything touches the GPU."""
import ctypes

import pytest
import torch

SA_OK, SA_ERR_NULL, SA_ERR_SHAPE, SA_ERR_UNSUPPORTED, SA_ERR_ALIGNMENT = 0, 1, 2, 3, 7
FAKE = ctypes.c_void_p(0x10000)       # aligned, never dereferenced: rejected first
MISALIGNED = ctypes.c_void_p(0x10008)
ODD = ctypes.c_void_p(0x10001)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from attention_softmax_sinks_gb300 import _build
    import attention_softmax_sinks_gb300 as sa
    _build.build()
    return sa.load_library()


@pytest.mark.parametrize("args,status", [
    ((FAKE, -1, 4, 8, FAKE, FAKE, FAKE), SA_ERR_SHAPE), ((FAKE, 5, 0, 8, FAKE, FAKE, FAKE), SA_ERR_SHAPE),
    ((FAKE, 5, 9, 8, FAKE, FAKE, FAKE), SA_ERR_SHAPE), ((FAKE, 5, 4, 0, FAKE, FAKE, FAKE), SA_ERR_SHAPE),
    ((FAKE, 5, 4, 257, FAKE, FAKE, FAKE), SA_ERR_SHAPE), ((FAKE, 2 ** 28, 8, 8, FAKE, FAKE, FAKE), SA_ERR_SHAPE),
    ((None, 5, 4, 8, FAKE, FAKE, FAKE), SA_ERR_NULL), ((FAKE, 5, 4, 8, None, FAKE, FAKE), SA_ERR_NULL),
    ((FAKE, 5, 4, 8, FAKE, None, FAKE), SA_ERR_NULL), ((FAKE, 5, 4, 8, FAKE, FAKE, None), SA_ERR_NULL),
    ((None, 0, 4, 8, None, None, None), SA_ERR_NULL),  # the offsets are written even then
])
def test_group_rows_rejects(lib, args, status):
    assert lib.moe_group_rows(*args, None) == status


@pytest.mark.parametrize("args,status", [
    ((FAKE, FAKE, FAKE, 8, -1, 4, 64, FAKE), SA_ERR_SHAPE), ((FAKE, FAKE, FAKE, -8, 2, 4, 64, FAKE), SA_ERR_SHAPE),
    ((FAKE, FAKE, FAKE, 8, 2, 0, 64, FAKE), SA_ERR_SHAPE), ((FAKE, FAKE, FAKE, 8, 2, 9, 64, FAKE), SA_ERR_SHAPE),
    ((FAKE, FAKE, FAKE, 8, 2, 4, 0, FAKE), SA_ERR_SHAPE), ((FAKE, FAKE, FAKE, 8, 2, 4, 60, FAKE), SA_ERR_UNSUPPORTED),
    ((FAKE, FAKE, FAKE, 8, 2 ** 30, 4, 2 ** 20, FAKE), SA_ERR_SHAPE),
    ((None, FAKE, FAKE, 8, 2, 4, 64, FAKE), SA_ERR_NULL), ((FAKE, None, FAKE, 8, 2, 4, 64, FAKE), SA_ERR_NULL),
    ((FAKE, FAKE, None, 8, 2, 4, 64, FAKE), SA_ERR_NULL), ((FAKE, FAKE, FAKE, 8, 2, 4, 64, None), SA_ERR_NULL),
    ((MISALIGNED, FAKE, FAKE, 8, 2, 4, 64, FAKE), SA_ERR_ALIGNMENT),
    ((FAKE, FAKE, FAKE, 8, 2, 4, 64, MISALIGNED), SA_ERR_ALIGNMENT),
    ((None, None, None, 0, 0, 4, 64, None), SA_OK),
])
def test_combine_rejects(lib, args, status):
    assert lib.moe_combine(*args, None) == status


def _grouped(lib, name, **kw):
    a = dict(x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, bias=FAKE, off=FAKE, tok=FAKE, x_rows=5, rows=9, e=4, n=64, k=64,
             alpha=1.702, limit=7.0, out=FAKE)
    a.update(kw)
    operands = [a["x"], a["xs"], a["w"], a["ws"]] if "mxfp4" in name else [a["x"], a["w"]]
    act = [a["alpha"], a["limit"]] if "swiglu" in name else []
    return getattr(lib, name)(*operands, a["bias"], a["off"], a["tok"], a["x_rows"], a["rows"], a["e"], a["n"], a["k"],
                              *act, a["out"], None)


GROUPED = ["grouped_linear_bias", "grouped_linear_swiglu", "grouped_mxfp4_linear_bias", "grouped_mxfp4_linear_swiglu"]


@pytest.mark.parametrize("name", GROUPED)
@pytest.mark.parametrize("kw,status", [
    (dict(x=None), SA_ERR_NULL), (dict(w=None), SA_ERR_NULL), (dict(off=None), SA_ERR_NULL),
    (dict(out=None), SA_ERR_NULL), (dict(rows=-1), SA_ERR_SHAPE), (dict(x_rows=-1), SA_ERR_SHAPE),
    (dict(rows=2 ** 30 + 1), SA_ERR_SHAPE), (dict(e=0), SA_ERR_SHAPE), (dict(e=257), SA_ERR_SHAPE),
    (dict(n=0), SA_ERR_SHAPE), (dict(k=0), SA_ERR_SHAPE), (dict(n=2 ** 30, e=4), SA_ERR_SHAPE),
    (dict(rows=2 ** 30, n=2 ** 20, e=1), SA_ERR_SHAPE),       # more tiles than are counted
    (dict(k=60), SA_ERR_UNSUPPORTED), (dict(tok=None), SA_ERR_SHAPE),  # 5 rows of x for 9 rows
    (dict(x_rows=0), SA_ERR_SHAPE), (dict(x=MISALIGNED), SA_ERR_ALIGNMENT), (dict(w=MISALIGNED), SA_ERR_ALIGNMENT),
    (dict(bias=ODD), SA_ERR_ALIGNMENT), (dict(out=ODD), SA_ERR_ALIGNMENT),
    (dict(rows=0), SA_OK), (dict(rows=0, x=None, w=None, off=None, out=None), SA_OK),
])
def test_grouped_products_reject(lib, name, kw, status):
    assert _grouped(lib, name, **kw) == status


@pytest.mark.parametrize("name", GROUPED[1::2])
@pytest.mark.parametrize("kw", [dict(n=63), dict(alpha=NAN), dict(alpha=INF), dict(limit=0.0), dict(limit=-1.0),
                                dict(limit=NAN)])
def test_swiglu_constants_rejected(lib, name, kw):
    assert _grouped(lib, name, **kw) == SA_ERR_SHAPE


@pytest.mark.parametrize("name", GROUPED[2:])
def test_grouped_mxfp4_scales_rejected(lib, name):
    assert _grouped(lib, name, xs=None) == SA_ERR_NULL
    assert _grouped(lib, name, ws=None) == SA_ERR_NULL
    assert _grouped(lib, name, xs=MISALIGNED) == SA_ERR_ALIGNMENT
    assert _grouped(lib, name, ws=MISALIGNED) == SA_ERR_ALIGNMENT
    assert _grouped(lib, name, k=72) == SA_ERR_UNSUPPORTED  # a multiple of 8, not of 32


def test_mxfp4_linear_and_conversions_reject(lib):
    f = lib.mxfp4_linear_bias
    assert f(FAKE, FAKE, FAKE, FAKE, None, -1, 64, 64, FAKE, None) == SA_ERR_SHAPE
    assert f(FAKE, FAKE, FAKE, FAKE, None, 4, 64, 48, FAKE, None) == SA_ERR_UNSUPPORTED
    assert f(FAKE, None, FAKE, FAKE, None, 4, 64, 64, FAKE, None) == SA_ERR_NULL
    assert f(None, None, None, None, None, 0, 64, 64, None, None) == SA_OK
    q, d = lib.mxfp4_quantize, lib.mxfp4_dequantize
    assert q(FAKE, 0, -1, 64, FAKE, FAKE, None) == SA_ERR_SHAPE
    assert q(FAKE, 0, 4, 0, FAKE, FAKE, None) == SA_ERR_SHAPE
    assert q(FAKE, 0, 2 ** 40, 64, FAKE, FAKE, None) == SA_ERR_SHAPE
    assert q(FAKE, 0, 4, 48, FAKE, FAKE, None) == SA_ERR_UNSUPPORTED
    assert q(None, 0, 4, 64, FAKE, FAKE, None) == SA_ERR_NULL
    assert q(FAKE, 1, 4, 64, FAKE, None, None) == SA_ERR_NULL
    assert q(MISALIGNED, 0, 4, 64, FAKE, FAKE, None) == SA_ERR_ALIGNMENT
    assert q(None, 0, 0, 64, None, None, None) == SA_OK
    assert d(FAKE, FAKE, -1, 64, FAKE, None) == SA_ERR_SHAPE
    assert d(FAKE, FAKE, 4, 40, FAKE, None) == SA_ERR_UNSUPPORTED
    assert d(FAKE, FAKE, 4, 64, None, None) == SA_ERR_NULL
    assert d(FAKE, MISALIGNED, 4, 64, FAKE, None) == SA_ERR_ALIGNMENT
    assert d(None, None, 0, 64, None, None) == SA_OK


def test_wrappers_refuse_what_is_not_a_cuda_tensor_of_the_right_kind():
    import attention_softmax_sinks_gb300 as sa
    x, i = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    w, off = torch.zeros(3, 32, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    u = torch.zeros(4, 32, dtype=torch.uint8)
    calls = [lambda: sa.moe_group_rows(i, 8), lambda: sa.moe_group_rows(None, 8),
             lambda: sa.moe_combine(x, i, i.to(torch.bfloat16)), lambda: sa.moe_combine(x, None, None),
             lambda: sa.grouped_linear_bias(x, w, off), lambda: sa.grouped_linear_swiglu(x, None, off),
             lambda: sa.mxfp4_quantize(x), lambda: sa.mxfp4_quantize(None), lambda: sa.mxfp4_quantize(x.half()),
             lambda: sa.mxfp4_dequantize(u, u), lambda: sa.mxfp4_dequantize(None, u),
             lambda: sa.mxfp4_linear_bias(u, u, u, u), lambda: sa.mxfp4_linear_bias(u, None, u, u),
             lambda: sa.grouped_mxfp4_linear_bias(u, None, w.to(torch.uint8), u, off)]
    for call in calls:
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        sa.grouped_linear_bias(x, x, off)  # w must have three dimensions


def test_scale_columns():
    import attention_softmax_sinks_gb300 as sa
    from oracle import experts
    for k in (32, 480, 512, 544, 2880, 4096, 5760):
        assert sa.mxfp4_scale_columns(k) == experts.scale_columns(k)
    assert [sa.mxfp4_scale_columns(k) for k in (32, 512, 544, 2880)] == [16, 16, 32, 96]


def test_index_arrays_at_odd_addresses_are_refused(lib):
    """int32 arrays need 4-byte addresses and bf16 weights 2-byte ones: the kernels' loads would fault."""
    two = ctypes.c_void_p(0x10002)
    good = (FAKE, 5, 4, 8, FAKE, FAKE, FAKE)
    for at in (0, 4, 5, 6):
        assert lib.moe_group_rows(*good[:at], two, *good[at + 1:], None) == SA_ERR_ALIGNMENT
    assert lib.moe_group_rows(None, 0, 4, 8, two, None, None, None) == SA_ERR_ALIGNMENT
    assert lib.moe_combine(FAKE, two, FAKE, 8, 2, 4, 64, FAKE, None) == SA_ERR_ALIGNMENT
    assert lib.moe_combine(FAKE, FAKE, ODD, 8, 2, 4, 64, FAKE, None) == SA_ERR_ALIGNMENT
    for name in GROUPED:
        assert _grouped(lib, name, off=two) == SA_ERR_ALIGNMENT
        assert _grouped(lib, name, tok=two) == SA_ERR_ALIGNMENT
