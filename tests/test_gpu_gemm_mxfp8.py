"""GPU tests of the MXFP8 x MXFP4 product against the exact product in 64 bits.

Tolerance: every product of two dequantized values is exact in FP32; only the K
additions round, |C - exact| <= (K + 2) 2^-22 (|A| |B|^T) (2^-22 and not 2^-24:
the tensor core aligns and truncates the addends of a step, as in the tests of
the 4-bit GEMMs), plus half a step of the output type."""
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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def tokens(M, K, seed):
    """Random finite E4M3 codes and scale bytes; the scale rows past M and the
    bytes of rows that do not exist hold 0xFF (NaN): they may not be used."""
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 256, (M, K), dtype=np.uint8)
    q[(q & 0x7F) == 0x7F] = 0x7E
    sf = np.full(-(-M // 128) * 128 * K // 32, 0xFF, np.uint8)
    sf[plain.scale_index(M, K // 32, True)] = rng.integers(118, 130, (M, K // 32))
    return q, sf


def weights(N, K, seed):
    rng = np.random.default_rng(seed)
    return (rng.integers(0, 256, (N, K // 2), dtype=np.uint8),
            rng.integers(116, 128, N * K // 32, dtype=np.uint8))


def check(c, qa, sfa, qb, sfb, half=0.0):
    a, b = plain.decode8(qa, sfa, True), plain.decode4(qb, sfb)
    exact, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    err = np.abs(c.double().cpu().numpy() - exact)
    bound = (a.shape[1] + 2) * 2.0 ** -22 * mag * (1 + half) + half * np.abs(exact) + 1e-30
    assert np.all(err <= bound), float(np.max(err / bound))


SHAPES = [(1, 128, 128), (1, 128, 4096), (2, 4096, 256), (16, 384, 640), (17, 256, 1280),
          (64, 128, 2176), (65, 256, 896), (128, 128, 128), (129, 384, 1152), (333, 512, 640),
          (1, 14336, 512), (257, 128, 384), (1030, 5120, 256)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_one_hot_weights_select_columns(M, N, K):
    """Each weight row has one code 1.0 with scale 2^0: C is a column selection
    of the dequantized tokens, exact in any order.  A misplaced code, scale byte
    or tile shows."""
    qa, sfa = tokens(M, K, 1)
    rng = np.random.default_rng(2)
    at = rng.integers(0, K, N)
    code = np.zeros((N, K), np.uint8)
    code[np.arange(N), at] = 2
    qb = code[:, 0::2] | code[:, 1::2] << 4
    sfb = np.full(N * K // 32, 127, np.uint8)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    c = fq.fp4q_gemm_mxfp8_mxfp4(dev(qa), dev(sfa), dev(qb), dev(sfb), status=status)
    assert int(status) == 0
    np.testing.assert_array_equal(c.double().cpu().numpy(), plain.decode8(qa, sfa, True)[:, at])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", SHAPES + [(3, 256, 14336), (64, 4096, 4096), (300, 2048, 2048)])
def test_random_codes_and_scales(M, N, K, dtype):
    (qa, sfa), (qb, sfb) = tokens(M, K, 3), weights(N, K, 4)
    args = [dev(a) for a in (qa, sfa, qb, sfb)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    c = fq.fp4q_gemm_mxfp8_mxfp4(*args, out_dtype=dtype, status=status)
    assert int(status) == 0
    check(c, qa, sfa, qb, sfb, 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2)
    assert torch.equal(c, fq.fp4q_gemm_mxfp8_mxfp4(*args, out_dtype=dtype))   # equal bits


@pytest.mark.parametrize("M", [1, 40, 100, 200])
def test_output_with_a_stride_and_its_surroundings(M):
    (qa, sfa), (qb, sfb) = tokens(M, 512, 5), weights(256, 512, 6)
    big = torch.full((M + 2, 320), 7.0, device=DEV)
    out = big[1:M + 1, 32:288]
    fq.fp4q_gemm_mxfp8_mxfp4(dev(qa), dev(sfa), dev(qb), dev(sfb), out=out)
    check(out, qa, sfa, qb, sfb)
    big[1:M + 1, 32:288] = 7.0
    assert (big == 7.0).all()


def test_empty_products():
    (qa, sfa), (qb, sfb) = tokens(3, 128, 7), weights(128, 128, 8)
    c = fq.fp4q_gemm_mxfp8_mxfp4(dev(qa)[:0], dev(sfa), dev(qb), dev(sfb))
    assert c.shape == (0, 128)
    c = fq.fp4q_gemm_mxfp8_mxfp4(dev(qa)[:, :0].contiguous(), dev(sfa), dev(qb)[:, :0].contiguous(),
                                 dev(sfb))
    assert c.shape == (3, 128) and not c.any()


def test_fprop_and_dgrad_of_a_linear_layer():
    """Norm -> MXFP8 -> product with W, and the input's gradient from the
    column-wise copy of W, through the library's quantizers."""
    g = torch.Generator().manual_seed(9)
    M, N, K = 200, 384, 512
    x = torch.randn(M, K, generator=g).bfloat16().to(DEV)
    w = (torch.randn(N, K, generator=g) * 0.05).bfloat16().to(DEV)
    dy = (torch.randn(M, N, generator=g) * 1e-2).bfloat16().to(DEV)
    sw = fq.SCALE_SWIZZLED
    qw = fq.fp4q_quantize_mxfp4(w, layouts=fq.ROWWISE | fq.COLWISE, scale_layout=sw)
    n = fq.fp4q_rmsnorm_mxfp8(x, torch.ones(K, device=DEV), scale_layout=sw)
    for act, q, sf in ((n, qw["q_row"], qw["sf_row"]),
                       (fq.fp4q_quantize_mxfp8(dy, scale_layout=sw), qw["q_col"], qw["sf_col"])):
        c = fq.fp4q_gemm_mxfp8_mxfp4(act["q"], act["sf"], q, sf)
        check(c, act["q"].cpu().numpy(), act["sf"].cpu().numpy(), q.cpu().numpy(), sf.cpu().numpy())


def test_captured_products_and_another_stream():
    shapes = [(1, 512, 2048), (200, 256, 512), (520, 5120, 256)]
    data = [[dev(a) for a in (*tokens(M, K, 20), *weights(N, K, 21))] for M, N, K in shapes]
    want = [fq.fp4q_gemm_mxfp8_mxfp4(*d) for d in data]
    static = [[torch.zeros_like(t) for t in d] for d in data]
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        outs = [fq.fp4q_gemm_mxfp8_mxfp4(*d) for d in static]
    for s, d in zip(static, data):
        for t, v in zip(s, d):
            t.copy_(v)
    gr.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [fq.fp4q_gemm_mxfp8_mxfp4(*d) for d in data]
    torch.cuda.synchronize()
    for a, b, c in zip(outs, again, want):
        assert torch.equal(a, c) and torch.equal(b, c)
