"""GPU tests of MXFP8: the quantizer and its decode, bit for bit against the
plain form in 64 bits (every step rounds once, so the codes are fixed)."""
import numpy as np
import pytest
import torch

import fp4_block_scaled_04_b200 as fq
import plain_mxfp8 as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fq.lib()


def values(rows, cols, seed, dtype):
    """Normal values, blocks of many magnitudes, a zero block, signed zeros,
    maxima at the scale's borders."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, cols // 32)).repeat(32, 1))
    x = torch.from_numpy(x.astype(np.float32))
    b = x.view(rows, cols // 32, 32)
    b[0, 0] = 0
    b[0, 0, 3] = -0.0
    for i, m in enumerate([448.0, 256.0, 512.0, 449.0, 447.0, 672.0, 336.0, 2.0 ** -126, 3e38]):
        if rows * (cols // 32) > i + 1:
            r, c = divmod(i + 1, cols // 32)
            b[r, c].clamp_(-m, m)
            b[r, c, i] = m
    return x.to(dtype)


@pytest.mark.parametrize("swizzled", [False, True])
@pytest.mark.parametrize("mode", [plain.RNE, plain.CEIL, plain.FLOOR])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 4096), (3, 96), (130, 160), (257, 1120)])
def test_quantize_bit_exact(rows, cols, dtype, mode, swizzled):
    x = values(rows, cols, rows + cols, dtype)
    layout = fq.SCALE_SWIZZLED if swizzled else fq.SCALE_LINEAR
    out = fq.fp4q_quantize_mxfp8(x.to(DEV), e8m0_mode=mode, scale_layout=layout)
    want, e = plain.quantize(x.double().numpy(), mode)
    q, sf = out["q"].cpu().numpy(), out["sf"].cpu().numpy()
    np.testing.assert_array_equal(plain.e4m3_values(q), want)
    assert np.array_equal(np.signbit(plain.e4m3_values(q))[want != 0], np.signbit(want)[want != 0])
    at = plain.scale_index(rows, cols // 32, swizzled)
    np.testing.assert_array_equal(sf[at], e + 127)
    pad = np.ones(sf.size, bool)
    pad[at.reshape(-1)] = False
    assert not sf[pad].any()                            # padding bytes are 0
    for dt in (torch.float32, torch.bfloat16):
        y = fq.fp4q_dequantize(fq.FMT_MXFP8, out["q"], out["sf"], rows, cols, 1, 32,
                               scale_layout=layout, out_dtype=dt)
        exact = torch.from_numpy(want * np.repeat(np.ldexp(1.0, e), 32, 1))
        assert torch.equal(y.cpu(), exact.float().to(dt))


def test_quantize_rows_of_a_wider_matrix_and_guard_bytes():
    """A column range of a wider matrix, preallocated outputs inside larger
    buffers: nothing outside is written."""
    big = values(77, 512, 5, torch.bfloat16).to(DEV)
    x = big[:, 128:352]
    n = fq.fp4q_scale_bytes(77, 224, 32, fq.SCALE_SWIZZLED)
    qb = torch.full((77 * 224 + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    sb = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    out = {"q": qb[32:32 + 77 * 224].view(77, 224), "sf": sb[32:32 + n]}
    got = fq.fp4q_quantize_mxfp8(x, scale_layout=fq.SCALE_SWIZZLED, out=out)
    ref = fq.fp4q_quantize_mxfp8(x.contiguous(), scale_layout=fq.SCALE_SWIZZLED)
    assert torch.equal(got["q"], ref["q"]) and torch.equal(got["sf"], ref["sf"])
    for b in (qb, sb):
        assert (b[:32] == 0xA5).all() and (b[-32:] == 0xA5).all()


def test_empty_and_another_stream():
    out = fq.fp4q_quantize_mxfp8(torch.empty(0, 64, device=DEV))
    assert out["q"].shape == (0, 64) and out["sf"].numel() == 0
    x = values(300, 4096, 9, torch.float32).to(DEV)
    ref = fq.fp4q_quantize_mxfp8(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = fq.fp4q_quantize_mxfp8(x)
    s.synchronize()
    assert torch.equal(got["q"], ref["q"]) and torch.equal(got["sf"], ref["sf"])


def test_binding_refuses_what_does_not_fit():
    """The Python calls' own checks: shapes, types, devices and densities of outputs."""
    x = torch.zeros(4, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    q, sf = torch.empty(4, 64, dtype=torch.uint8, device=DEV), torch.empty(8, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        fq.fp4q_quantize_mxfp8(x.cpu())
    with pytest.raises(ValueError):
        fq.fp4q_quantize_mxfp8(x.t())                    # columns without unit stride
    with pytest.raises(TypeError):
        fq.fp4q_quantize_mxfp8(x.half())
    for bad in (q[:3], q.cpu(), torch.empty(4, 128, dtype=torch.uint8, device=DEV)[:, ::2]):
        with pytest.raises(ValueError):
            fq.fp4q_quantize_mxfp8(x, out={"q": bad, "sf": sf})
    with pytest.raises(TypeError):
        fq.fp4q_quantize_mxfp8(x, out={"q": q.view(torch.int8), "sf": sf})
    with pytest.raises(ValueError):
        fq.fp4q_quantize_mxfp8(x, out={"q": q, "sf": sf[:7]})
    with pytest.raises(fq.Fp4qError):
        fq.fp4q_quantize_mxfp8(torch.zeros(4, 48, device=DEV))
    with pytest.raises(ValueError):
        fq.fp4q_rmsnorm_mxfp8(x, w[:32])
    with pytest.raises(ValueError):
        fq.fp4q_rmsnorm_mxfp8(x, w, residual=x[:2])
    with pytest.raises(ValueError):
        fq.fp4q_rmsnorm_backward(x, x, w, torch.ones(3, device=DEV))
    with pytest.raises(ValueError):
        fq.fp4q_gemm_mxfp8_mxfp4(q, sf, q, sf)           # K of the weights
    wq = torch.zeros(128, 64, dtype=torch.uint8, device=DEV)
    xq = torch.zeros(4, 128, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        fq.fp4q_gemm_mxfp8_mxfp4(xq, sf, wq, torch.zeros(512, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        fq.fp4q_gemm_mxfp8_mxfp4(xq, torch.zeros(512, dtype=torch.uint8, device=DEV), wq,
                                 torch.zeros(512, dtype=torch.uint8, device=DEV),
                                 out=torch.empty(4, 64, device=DEV))
