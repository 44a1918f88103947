"""GPU tests of NaN and infinities in the MXFP8 calls: what they do to their own block,
row or token, and that nothing else changes by a bit."""
import numpy as np
import pytest
import torch

import fp4_block_scaled_04_b200 as fq

pytestmark = pytest.mark.gpu
DEV = "cuda"
SW = fq.SCALE_SWIZZLED
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fq.lib()


def randn(*shape, seed=0, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


@pytest.mark.parametrize("mode", [fq.E8M0_RNE, fq.E8M0_CEIL, fq.E8M0_OCP_FLOOR])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize(dtype, mode):
    """A NaN stays one and does not enter its block's scale; an infinity takes the largest
    scale of the mode, saturates, and decodes as itself."""
    x = randn(5, 256, seed=1, dtype=dtype)
    want = fq.fp4q_quantize_mxfp8(x, e8m0_mode=mode)
    x[1, 3], x[1, 40], x[2, 64:96] = NAN, -NAN, NAN
    x[3, 5], x[3, 133], x[4, 0], x[4, 1] = INF, -INF, INF, NAN
    got = fq.fp4q_quantize_mxfp8(x, e8m0_mode=mode)
    y = fq.fp4q_dequantize(fq.FMT_MXFP8, got["q"], got["sf"], 5, 256, 1, 32)
    assert torch.equal(torch.isnan(y), torch.isnan(x))
    assert torch.equal(y[torch.isinf(x)], x[torch.isinf(x)].float())
    touched = torch.zeros(5, 8, dtype=torch.bool, device=DEV)
    for r, b in ((1, 0), (1, 1), (2, 2), (3, 0), (3, 4), (4, 0)):
        touched[r, b] = True
    sf, old = got["sf"].view(5, 8), want["sf"].view(5, 8)
    assert torch.equal(sf[~touched], old[~touched])
    same = ~touched.repeat_interleave(32, 1)
    assert torch.equal(got["q"][same], want["q"][same])
    # the NaN's neighbours as without it (zero in its place)
    for r, at in ((1, 3), (1, 40)):
        b = at // 32
        clean = x[r:r + 1, 32 * b:32 * b + 32].clone()
        clean[0, at % 32] = 0
        ref = fq.fp4q_quantize_mxfp8(clean, e8m0_mode=mode)
        assert int(sf[r, b]) == int(ref["sf"][0])
        keep = torch.arange(32, device=DEV) != at % 32
        assert torch.equal(got["q"][r, 32 * b:32 * b + 32][keep], ref["q"][0][keep])
    assert int(sf[2, 2]) == 0
    top = 247 if mode == fq.E8M0_OCP_FLOOR else 254
    assert int(sf[3, 0]) == int(sf[3, 4]) == int(sf[4, 0]) == top


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(6, 96), (9, 4096), (1300, 1056), (400, 4096), (300, 10240)])
def test_norm(rows, cols, dtype):
    """A row with a NaN has rstd and codes NaN; one with an infinity has rstd 0, NaN in the
    infinity's place and zeros beside it."""
    x, r = randn(rows, cols, seed=2, dtype=dtype), randn(rows, cols, seed=3, dtype=dtype)
    w = 1 + 0.2 * randn(cols, seed=4)
    want = fq.fp4q_rmsnorm_mxfp8(x, w, residual=r, want_y=True)
    x[1, 7], x[3, cols - 1], x[4, 0], r[4, 0] = NAN, INF, INF, -INF
    got = fq.fp4q_rmsnorm_mxfp8(x, w, residual=r, want_y=True)
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[[1, 3, 4]] = False
    for k in ("q", "rstd", "sum", "y"):
        assert torch.equal(got[k][keep], want[k][keep]), k
    assert torch.equal(got["sf"].view(rows, -1)[keep], want["sf"].view(rows, -1)[keep])
    for row in (1, 4):
        assert torch.isnan(got["rstd"][row]) and torch.isnan(got["y"][row]).all()
        assert ((got["q"][row] & 0x7F) == 0x7F).all()
    assert float(got["rstd"][3]) == 0
    assert torch.isnan(got["y"][3, -1]) and not got["y"][3, :-1].float().any()
    assert (got["q"][3, -1] & 0x7F) == 0x7F and not (got["q"][3, :-1] & 0x7F).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(6, 96), (9, 4096), (1300, 1056), (400, 4096)])
def test_norm_backward(rows, cols, dtype):
    """A NaN in the gradient makes its row of dx NaN and its column of dweight."""
    s, g = randn(rows, cols, seed=5, dtype=dtype), randn(rows, cols, seed=6, dtype=dtype)
    w = 1 + 0.2 * randn(cols, seed=7)
    rstd = fq.fp4q_rmsnorm_mxfp8(s, w)["rstd"]
    want = fq.fp4q_rmsnorm_backward(g, s, w, rstd, dsum=s)
    g[2, 5] = NAN
    got = fq.fp4q_rmsnorm_backward(g, s, w, rstd, dsum=s)
    keep = torch.arange(rows, device=DEV) != 2
    assert torch.equal(got["dx"][keep], want["dx"][keep]) and torch.isnan(got["dx"][2]).all()
    keep = torch.arange(cols, device=DEV) != 5
    assert torch.equal(got["dweight"][keep], want["dweight"][keep])
    assert torch.isnan(got["dweight"][5])


@pytest.mark.parametrize("M", [3, 40, 100, 300])
def test_product(M):
    """A token with a NaN or an infinity: its row alone is affected."""
    x = randn(M, 512, seed=8)
    w = fq.fp4q_quantize_mxfp4(randn(384, 512, seed=9), scale_layout=SW)

    def product():
        q = fq.fp4q_quantize_mxfp8(x, scale_layout=SW)
        return fq.fp4q_gemm_mxfp8_mxfp4(q["q"], q["sf"], w["q_row"], w["sf_row"])

    want = product()
    x[0, 100], x[2, 511] = NAN, INF
    got = product()
    keep = [i for i in range(M) if i not in (0, 2)]
    assert torch.equal(got[keep], want[keep])
    assert torch.isnan(got[0]).all() and not torch.isfinite(got[2]).all()


@pytest.mark.parametrize("T", [3, 16, 24, 64])
def test_expert_layer(T):
    """A token with a NaN alone gets NaN.  A router row with +inf chooses no expert, as one
    without a finite logit does: its output is 0, and the others' stay what they are."""
    E, H, I = 8, 256, 256
    x, logits = randn(T, H, seed=10), randn(T, E, seed=11)
    q13 = fq.fp4q_quantize_mxfp4(randn(E * 2 * I, H, seed=12) * 0.1, scale_layout=SW)
    q2 = fq.fp4q_quantize_mxfp4(randn(E * H, I, seed=13) * 0.1, scale_layout=SW)

    def layer():
        q = fq.fp4q_quantize_mxfp8(x, scale_layout=SW)
        return fq.fp4q_moe_mxfp4(q["q"], q["sf"], logits, q13["q_row"].view(E, 2 * I, H // 2),
                                 q13["sf_row"], q2["q_row"].view(E, H, I // 2), q2["sf_row"],
                                 top_k=E, out_dtype=torch.float32)

    want = layer()
    x[1, 9] = NAN
    logits[0, 3] = INF
    got = layer()
    assert torch.isnan(got[1]).all() and not got[0].any()
    if T > 2:
        assert torch.equal(got[2:], want[2:])
    logits[0] = NAN
    assert not layer()[0].any()
