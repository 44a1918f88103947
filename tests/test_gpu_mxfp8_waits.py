"""Failure detection of the MXFP8 tensor-core kernels without a GPU fault: their test
hooks stop the loading warps after some K-tiles, so that a bounded wait (about 10 ms here)
runs out with copies and MMAs in flight.  The kernel has to report it through status, come
to its end, and leave the GPU so that the calls behind it are right."""
import pytest
import torch

import fp4_block_scaled_04_b200 as fq

pytestmark = pytest.mark.gpu
DEV = "cuda"
MANY = 1 << 40                                      # a loader that does not stop


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fq.lib()


def operands(M, N, K):
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    x = fq.fp4q_quantize_mxfp8(torch.randn(M, K, device=DEV, generator=g),
                               scale_layout=fq.SCALE_SWIZZLED)
    w = fq.fp4q_quantize_mxfp4(torch.randn(N, K, device=DEV, generator=g) * 0.05,
                               scale_layout=fq.SCALE_SWIZZLED)
    return x["q"], x["sf"], w["q_row"], w["sf_row"]


# (loads of the first and of the second loader); one loader up to 64 tokens
ONE = [(0, 0), (1, 0)]
# the CTAs of a pair stop together, and either one before the other
TWO = [(0, 0), (1, 1), (1, 0), (0, 1), (MANY, 0), (0, MANY)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K,loads", [
    *[(M, 256, 2048, ld) for M in (1, 40) for ld in ONE],           # K split over clusters
    *[(M, 40960, 1024, (n, 0)) for M in (1, 40) for n in (0, 3, 7, 11)],   # some CTAs with two tiles
    *[(300, 512, 2048, ld) for ld in TWO],                          # K split over pairs
    *[(100, 256, 4096, ld) for ld in TWO],
    *[(1030, 5120, 1024, ld) for ld in                              # some pairs with two tiles
      TWO + [(3, 5), (5, 3), (7, 2), (2, 8), (11, 9), (9, 11), (13, 13)]]])
def test_product(M, N, K, loads, dtype):
    args = operands(M, N, K)
    want = fq.fp4q_gemm_mxfp8_mxfp4(*args, out_dtype=dtype)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    later = torch.zeros(1, dtype=torch.int32, device=DEV)
    c = torch.empty_like(want)
    p = [t.data_ptr() for t in args]
    for _ in range(2):
        rc = fq.lib().fp4q_gemm_mxfp8_mxfp4_withhold_loads(
            *p, M, N, K, c.data_ptr(), 0 if dtype == torch.bfloat16 else 1, N, *loads,
            status.data_ptr(), fq._raw_stream(0))
        assert rc == 0
        # behind it without a pause
        got = fq.fp4q_gemm_mxfp8_mxfp4(*args, out_dtype=dtype, status=later)
        assert torch.equal(got, want)
        assert int(status) == 1 and int(later) == 0
        status.zero_()


# the loaders of weights and of tokens stop together, and either one before the other
LOADERS = [(0, 0), (2, 2), (3, 1), (1, 3), (MANY, 1), (1, MANY), (MANY, 0), (0, MANY)]


@pytest.mark.parametrize("product", [1, 2])
@pytest.mark.parametrize("loads", LOADERS)
@pytest.mark.parametrize("T,E,k,H,I", [
    (1, 8, 2, 1024, 4096), (13, 8, 2, 2048, 1024), (16, 64, 8, 1024, 1024),  # routing inside
    (24, 16, 4, 1024, 1024), (40, 16, 4, 1024, 1024), (64, 32, 8, 1024, 2048)])
def test_expert_layer(T, E, k, H, I, loads, product):
    g = torch.Generator(device=DEV).manual_seed(T)

    def w4(rows, cols):
        o = fq.fp4q_quantize_mxfp4(torch.randn(rows, cols, device=DEV, generator=g) * 0.05,
                                   scale_layout=fq.SCALE_SWIZZLED)
        return o["q_row"], o["sf_row"]

    (q13, s13), (q2, s2) = w4(E * 2 * I, H), w4(E * H, I)
    x = fq.fp4q_quantize_mxfp8(torch.randn(T, H, device=DEV, generator=g),
                               scale_layout=fq.SCALE_SWIZZLED)
    logits = torch.randn(T, E, device=DEV, generator=g)
    args = (x["q"], x["sf"], logits, q13.view(E, 2 * I, H // 2), s13, q2.view(E, H, I // 2), s2)
    want = fq.fp4q_moe_mxfp4(*args, top_k=k)
    need = fq.lib().fp4q_moe_mxfp4_workspace_bytes(T, E, k, H, I)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    later = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.empty_like(want)
    p = [t.data_ptr() for t in args]
    for _ in range(2):
        rc = fq.lib().fp4q_moe_mxfp4_withhold_loads(
            *p[:3], 1, *p[3:], T, E, k, H, I, 1, out.data_ptr(), 0, H, ws.data_ptr(), need,
            product, *loads, status.data_ptr(), fq._raw_stream(0))
        assert rc == 0
        # behind it without a pause, in the same workspace
        got = fq.fp4q_moe_mxfp4(*args, top_k=k, workspace=ws, status=later)
        assert torch.equal(got, want)
        assert int(status) == 1 and int(later) == 0
        status.zero_()
