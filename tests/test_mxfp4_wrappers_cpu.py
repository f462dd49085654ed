"""Argument marshalling of the MXFP4 conversions for sizes that no test machine holds: tensors
without memory (on the meta device) and a library that records its arguments."""
import pytest
import torch


class Recorder:
    def __getattr__(self, name):
        return lambda *args: self.__dict__.setdefault("calls", []).append((name, args)) or 0


@pytest.fixture
def recorded(monkeypatch):
    import attention_softmax_sinks_gb300 as sa
    lib = Recorder()
    monkeypatch.setattr(sa, "load_library", lambda: lib)
    monkeypatch.setattr(sa, "_call", lambda fn, dev, stream, *args: fn(*args))

    def kind(t, name, dtype):  # _dev without the demand for CUDA
        if not isinstance(t, torch.Tensor) or t.dtype != dtype:
            raise TypeError(name)
        if not t.is_contiguous():
            raise ValueError(name)
        return t

    monkeypatch.setattr(sa, "_dev", kind)
    return sa, lib


@pytest.mark.parametrize("lead", [(2 ** 31,), (2 ** 32 + 5,), (3, 2 ** 31), (7,), ()])
def test_what_quantize_returns_dequantize_takes(recorded, lead):
    """Any number of rows (rows * K < 2^40): the row count is 64 bits wide in both calls."""
    sa, lib = recorded
    rows = torch.Size(lead).numel()
    x = torch.empty((*lead, 96), dtype=torch.bfloat16, device="meta")
    codes, scales = sa.mxfp4_quantize(x)
    assert codes.shape == (*lead, 48) and scales.shape == (*lead, 16)
    out = sa.mxfp4_dequantize(codes, scales)
    assert out.shape == x.shape and out.dtype is torch.bfloat16
    (_, q), (_, d) = lib.calls
    assert q[2:4] == (rows, 96) and d[2:4] == (rows, 96)


def test_dequantize_refuses_what_does_not_fit(recorded):
    sa, lib = recorded
    u8 = lambda *shape: torch.empty(shape, dtype=torch.uint8, device="meta")  # noqa: E731
    for codes, scales in ((u8(2, 2 ** 30), u8(2, 2 ** 26)), (u8(5, 48), u8(5, 32)), (u8(5, 48), u8(4, 16)),
                          (u8(5, 48), u8(80)), (u8(), u8(16)), (u8(48, 5).t(), u8(5, 16))):
        with pytest.raises(ValueError):
            sa.mxfp4_dequantize(codes, scales)
    for codes, scales in ((None, u8(5, 16)), (u8(5, 48), None), (u8(5, 48), u8(5, 16).to(torch.int8))):
        with pytest.raises(TypeError):
            sa.mxfp4_dequantize(codes, scales)
    assert "calls" not in lib.__dict__
