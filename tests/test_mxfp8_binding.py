"""The Python binding's own checks of the MXFP8 calls, on the CPU: tensors without
memory stand for device tensors, and the library's entry points only count calls, so a
call that would read or write past a buffer shows without running."""
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import fp4_block_scaled_04_b200 as fq

BF16, FP32, U8 = torch.bfloat16, torch.float32, torch.uint8


class Library:
    """Entry points that record their arguments and answer 0."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append((name, args))
            return 0
        return entry


@pytest.fixture
def L(monkeypatch):
    lib = Library()
    monkeypatch.setattr(fq, "lib", lambda: lib)
    monkeypatch.setattr(fq, "_stream", lambda device: None)
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")            # addresses of tensors without memory
        yield lib


def dev(*shape, dtype=U8, device="cuda:0"):
    return torch.empty(shape, dtype=dtype, device=device)


def dequantize(rows=1, cols=4096, q=None, sf=None, layout=fq.SCALE_SWIZZLED, **kw):
    q = dev(rows, cols) if q is None else q
    sf = dev(fq._mx_scale_bytes(rows, cols, layout)) if sf is None else sf
    return fq.fp4q_dequantize(fq.FMT_MXFP8, q, sf, rows, cols, 1, 32, scale_layout=layout, **kw)


def test_dequantize_takes_what_the_quantizer_gives(L):
    for layout in (fq.SCALE_LINEAR, fq.SCALE_SWIZZLED):
        for dt in (BF16, FP32):
            assert dequantize(layout=layout, out_dtype=dt).dtype == dt
    dequantize(q=dev(4096, dtype=torch.float8_e4m3fn), sf=dev(5000 * 4), out=dev(4096, dtype=FP32))
    dequantize(rows=0)
    assert len(L.calls) == 6


def test_dequantize_refuses_scales_of_the_other_layout(L):
    """One row of 4096: 128 scale bytes in rows, 16384 in padded tiles.  Taken for the
    other layout, a short buffer would be read far past its end."""
    with pytest.raises(ValueError):
        dequantize(sf=dev(128))
    with pytest.raises(ValueError):
        dequantize(rows=130, cols=64, sf=dev(130 * 2))
    assert not L.calls


@pytest.mark.parametrize("bad", [
    dict(q=lambda: dev(1, 4095)), dict(q=lambda: dev(4096, 2)[:, 0]),
    dict(sf=lambda: dev(16383)), dict(sf=lambda: dev(2 * 16384)[::2]),
    dict(sf=lambda: dev(16384, device="cpu")), dict(sf=lambda: dev(16384, device="cuda:1")),
    dict(out=lambda: dev(1, 4095, dtype=FP32)), dict(out=lambda: dev(4096, 2, dtype=FP32)[:, 0]),
    dict(out=lambda: dev(1, 4096, dtype=FP32, device="cpu")),
    dict(out=lambda: dev(1, 4096, dtype=FP32, device="cuda:1"))])
def test_dequantize_refuses_buffers_that_do_not_fit(L, bad):
    with pytest.raises(ValueError):
        dequantize(**{k: v() for k, v in bad.items()})
    assert not L.calls


@pytest.mark.parametrize("bad", [dict(out=torch.float16), dict(out=torch.float64),
                                 dict(out_dtype=torch.float16), dict(q=torch.int16),
                                 dict(sf=torch.int32)])
def test_dequantize_refuses_types(L, bad):
    """An output of another type would be written as FP32: past its end where its
    elements are smaller."""
    kw = {k: v if k == "out_dtype" else dev(1 if k == "q" else 16384, 4096, dtype=v)
          for k, v in bad.items()}
    with pytest.raises(TypeError):
        dequantize(**kw)
    assert not L.calls


def test_scale_bytes_as_the_library_counts_them():
    """The binding's count of scale bytes is the library's."""
    for layout in (fq.SCALE_LINEAR, fq.SCALE_SWIZZLED):
        for rows in (0, 1, 127, 128, 129, 8192):
            for cols in (32, 64, 96, 128, 160, 4096, 14336):
                want = fq.fp4q_scale_bytes(rows, cols, 32, layout)
                assert fq._mx_scale_bytes(rows, cols, layout) == want
