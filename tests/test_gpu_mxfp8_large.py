"""The MXFP8 calls where offsets pass 2^31 elements: the 64-bit index paths, against the
plain forms in 64 bits on rows and bands at the start, in the middle and at the end."""
import numpy as np
import pytest
import torch

import fp4_block_scaled_04_b200 as fq
import plain_mxfp8 as plain
from test_gpu_gemm_mxfp8 import tokens, weights
from test_gpu_rmsnorm import check_forward

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _need_room():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 60 * 2**30:
        pytest.skip("needs 60 GB of free device memory")
    fq.lib()
    yield
    torch.cuda.empty_cache()


def randn(rows, cols, seed, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn((rows, cols), generator=g, dtype=dtype, device=DEV)


@pytest.mark.parametrize("swizzled", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_and_dequantize(dtype, swizzled):
    R, C = 32769, 65568
    assert R * C > 2**31
    x = randn(R, C, 1, dtype)
    layout = fq.SCALE_SWIZZLED if swizzled else fq.SCALE_LINEAR
    out = fq.fp4q_quantize_mxfp8(x, scale_layout=layout)
    rows = [0, 1, R // 2 + 3, R - 1]
    want, e = plain.quantize(x[rows].double().cpu().numpy())
    np.testing.assert_array_equal(plain.e4m3_values(out["q"][rows].cpu().numpy()), want)
    at = torch.from_numpy(plain.scale_index(R, C // 32, swizzled)[rows]).to(DEV)
    np.testing.assert_array_equal(out["sf"].view(-1)[at].cpu().numpy(), e + 127)
    del x
    y = fq.fp4q_dequantize(fq.FMT_MXFP8, out["q"], out["sf"], R, C, 1, 32, scale_layout=layout,
                           out_dtype=dtype)
    exact = torch.from_numpy(want * np.repeat(np.ldexp(1.0, e), 32, 1)).float().to(dtype)
    assert torch.equal(y[rows].cpu(), exact)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm(dtype):
    R, C = 520293, 4128
    assert R * C > 2**31
    x = randn(R, C, 2, dtype)
    w = 1 + 0.2 * randn(1, C, 3, torch.float32)[0]
    out = fq.fp4q_rmsnorm_mxfp8(x, w)
    rows = [0, 1, R // 2 + 3, R - 2, R - 1]
    some = {"rstd": out["rstd"][rows], "q": out["q"][rows], "sf": out["sf"].view(R, -1)[rows]}
    check_forward({**some, "sf": some["sf"].reshape(-1)}, x[rows], w, 1e-6, False)
    del out["q"]
    g = randn(R, C, 4, dtype)
    got = fq.fp4q_rmsnorm_backward(g, x, w, out["rstd"])
    G, S, W, r = g[rows].double(), x[rows].double(), w.double(), out["rstd"][rows].double()[:, None]
    dx = r * (W * G - S * r * r * (W * G * S).mean(1, keepdim=True))
    mag = (r * W * G).abs() + S.abs() * r ** 3 * (W * G * S).abs().mean(1, keepdim=True)
    half = torch.finfo(dtype).eps / 2
    assert bool(((got["dx"][rows].double() - dx).abs()
                 <= 80 * U * mag + half * dx.abs() * 1.01).all())
    dw, mag = torch.zeros(C, dtype=torch.float64, device=DEV), torch.zeros(C, device=DEV)
    for i in range(0, R, 1 << 16):
        part = (g[i:i + (1 << 16)].float() * x[i:i + (1 << 16)].float()
                * out["rstd"][i:i + (1 << 16), None])
        dw += part.sum(0, dtype=torch.float64)
        mag += part.abs().sum(0)
    # a CTA's part adds the rows of at most a 148th of the matrix one by one, then at most
    # 592 parts are added; two products a row here and there
    assert bool(((got["dweight"].double() - dw).abs() <= (R // 148 + 600) * U * mag).all())


@pytest.mark.parametrize("M,ld,dtype", [(3, 1 << 30, torch.float32), (3, 1 << 30, torch.bfloat16),
                                        (40, 1 << 26, torch.bfloat16), (100, 1 << 25, torch.bfloat16),
                                        (300, 1 << 23, torch.float32)])
def test_product_with_far_rows(M, ld, dtype):
    """Few tokens whose output rows lie far apart."""
    N, K = 512, 640
    (qa, sfa), (qb, sfb) = tokens(M, K, 5), weights(N, K, 6)
    big = torch.empty(ld * (M - 1) + N, dtype=dtype, device=DEV)
    assert big.numel() > 2**31
    out = big.as_strided((M, N), (ld, 1))
    args = [torch.from_numpy(a).to(DEV) for a in (qa, sfa, qb, sfb)]
    fq.fp4q_gemm_mxfp8_mxfp4(*args, out=out)
    assert torch.equal(out, fq.fp4q_gemm_mxfp8_mxfp4(*args, out_dtype=dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product_of_many_tokens(dtype):
    M, N, K = 65601, 32896, 128
    assert M * N > 2**31
    (qa, sfa), (qb, sfb) = tokens(M, K, 7), weights(N, K, 8)
    c = fq.fp4q_gemm_mxfp8_mxfp4(*[torch.from_numpy(a).to(DEV) for a in (qa, sfa, qb, sfb)],
                                 out_dtype=dtype)
    rows = [0, 1, 255, 256, M // 2, M - 130, M - 1]
    a, b = plain.decode8(qa, sfa, True)[rows], plain.decode4(qb, sfb)
    exact, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    half = 0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2
    err = np.abs(c[rows].double().cpu().numpy() - exact)
    assert np.all(err <= (K + 2) * 2.0 ** -22 * mag * (1 + half) + half * np.abs(exact) + 1e-30)


def test_experts_far_apart():
    """256 experts of 2^24 values in W13: the first, the last and two between give the bits
    that they give as the only ones.  Equal logits of four: every weight is 1/4."""
    E, H, I = 256, 4096, 2048
    g = torch.Generator(device=DEV).manual_seed(9)
    q13 = torch.randint(0, 256, (E, 2 * I, H // 2), dtype=torch.uint8, device=DEV, generator=g)
    s13 = torch.randint(119, 122, (E, 2 * I * H // 32), dtype=torch.uint8, device=DEV, generator=g)
    q2 = torch.randint(0, 256, (E, H, I // 2), dtype=torch.uint8, device=DEV, generator=g)
    s2 = torch.randint(119, 122, (E, H * I // 32), dtype=torch.uint8, device=DEV, generator=g)
    assert q13.numel() * 2 > 2**31
    x = fq.fp4q_quantize_mxfp8(torch.randn(1, H, device=DEV, generator=g),
                               scale_layout=fq.SCALE_SWIZZLED)
    at = [0, 100, 201, 255]
    logits = torch.full((1, E), -float("inf"), device=DEV)
    logits[0, at] = 0.25
    got = fq.fp4q_moe_mxfp4(x["q"], x["sf"], logits, q13, s13.view(-1), q2, s2.view(-1), top_k=4,
                            out_dtype=torch.float32)
    ref = fq.fp4q_moe_mxfp4(x["q"], x["sf"], logits[:, at].contiguous(), q13[at], s13[at].view(-1),
                            q2[at], s2[at].view(-1), top_k=4, out_dtype=torch.float32)
    assert bool(got.any()) and torch.equal(got, ref)
