"""GPU tests of the mixture-of-experts layer against its definition in 64 bits.

Tolerance.  The two products accumulate in FP32 (2^-22 per addition, as for the
plain product); the sums over experts, the weights p (exp, a division, a
division by the sum: below 16 units of 2^-24) and the K additions give
(H + I + E + 64) 2^-22 of the magnitudes |p| |h| |W2|, times 4 for what the first
product's error does to h through the activation.  h is rounded to E4M3: where
the FP32 h and the exact h lie on two sides of a rounding border one code of h
moves by one step, 2^-3 relative at most.  Such borders are hit by chance of
about the FP32 error over the step (1e-5 per code), so up to two moved codes are
allowed for per output, each of at most p 2^-3 max|h| max|W2|."""
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


class Layer:
    """Random weights of one layer, on the host and on the device."""

    def __init__(self, E, H, I, seed):
        rng = np.random.default_rng(seed)
        self.E, self.H, self.I = E, H, I
        self.q13 = rng.integers(0, 256, (E, 2 * I, H // 2), dtype=np.uint8)
        self.s13 = rng.integers(119, 122, E * 2 * I * H // 32, dtype=np.uint8)
        self.q2 = rng.integers(0, 256, (E, H, I // 2), dtype=np.uint8)
        self.s2 = rng.integers(119, 122, E * H * I // 32, dtype=np.uint8)
        self.dev = [torch.from_numpy(a).to(DEV) for a in (self.q13, self.s13, self.q2, self.s2)]

    def w13(self, e):
        return plain.decode4(self.q13[e], self.s13.reshape(self.E, -1)[e])

    def w2(self, e):
        return plain.decode4(self.q2[e], self.s2.reshape(self.E, -1)[e])


def tokens(T, H, seed):
    g = torch.Generator().manual_seed(seed)
    out = fq.fp4q_quantize_mxfp8(torch.randn(T, H, generator=g).to(DEV),
                                 scale_layout=fq.SCALE_SWIZZLED)
    x = plain.decode8(out["q"].cpu().numpy(), out["sf"].cpu().numpy(), True)
    return out, x


def check(got, L, x, logits, k, renormalize):
    p = plain.route(logits.double().cpu().numpy(), k, renormalize)
    out, mag, flip = plain.moe(x, p, L.w13, L.w2)
    half = 0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    err = np.abs(got.double().cpu().numpy() - out)
    bound = 4 * (L.H + L.I + L.E + 64) * 2.0 ** -22 * mag + 2 * flip + half * np.abs(out) * 1.01
    # what the moved codes may explain is rare: nearly all outputs are without it
    tight = bound - 2 * flip + 1e-30
    assert np.all(err <= bound + 1e-30), float(np.max(err / (bound + 1e-30)))
    rows = np.abs(p).sum(1) > 0
    if rows.any():
        assert np.mean(err[rows] <= tight[rows]) > 0.5
    assert not got[torch.from_numpy(~rows)].any()


CASES = [  # T, E, k, H, I
    (1, 1, 1, 128, 128), (1, 8, 2, 256, 128), (1, 64, 8, 1024, 512), (3, 5, 3, 384, 256),
    (13, 8, 2, 2048, 1024), (16, 2, 2, 128, 640), (17, 40, 6, 512, 384), (31, 256, 16, 256, 128),
    (33, 12, 1, 640, 256), (64, 16, 4, 512, 512), (64, 4, 4, 1152, 128), (40, 33, 8, 4096, 128)]


@pytest.mark.parametrize("renormalize,dtype", [(True, torch.bfloat16), (False, torch.float32)])
@pytest.mark.parametrize("T,E,k,H,I", CASES)
def test_layer(T, E, k, H, I, renormalize, dtype):
    L = Layer(E, H, I, T + E)
    xq, x = tokens(T, H, 1)
    g = torch.Generator().manual_seed(2)
    logits = (torch.randn(T, E, generator=g) * 2).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = fq.fp4q_moe_mxfp4(xq["q"], xq["sf"], logits, *L.dev, top_k=k, renormalize=renormalize,
                            out_dtype=dtype, status=status)
    assert int(status) == 0
    check(got, L, x, logits, k, renormalize)
    again = fq.fp4q_moe_mxfp4(xq["q"], xq["sf"], logits, *L.dev, top_k=k,
                              renormalize=renormalize, out_dtype=dtype)
    assert torch.equal(got, again)


def test_masks_ties_and_bf16_logits():
    """Rows with no expert left, with fewer than k, with NaN; equal logits; all
    tokens on one expert."""
    L = Layer(40, 256, 256, 3)
    xq, x = tokens(40, 256, 4)
    inf = float("inf")
    logits = torch.randn(40, 40, generator=torch.Generator().manual_seed(5)).bfloat16().float()
    logits[0] = -inf
    logits[1, 1:] = -inf
    logits[2] = float("nan")
    logits[3, ::2] = float("nan")
    logits[4] = 0.0
    logits[5] = torch.finfo(torch.float32).min
    logits[6, 7] = 200.0                              # the others' probability underflows
    logits[8:, 33] = 30.0
    for t in (logits.to(DEV), logits.bfloat16().to(DEV)):
        for renorm in (True, False):
            got = fq.fp4q_moe_mxfp4(xq["q"], xq["sf"], t, *L.dev, top_k=4, renormalize=renorm,
                                    out_dtype=torch.float32)
            check(got, L, x, t, 4, renorm)


@pytest.mark.parametrize("T", [3, 20])
def test_zeros_of_either_sign_tie(T):
    """-0 and 0 are equal logits: the lowest indices are chosen, whatever the signs."""
    L = Layer(40, 256, 256, 13)
    xq, x = tokens(T, 256, 14)
    logits = torch.zeros(T, 40)
    logits[:, :24] = -0.0
    logits[1, 3::7] = 0.0
    for t in (logits.to(DEV), logits.bfloat16().to(DEV)):
        got = fq.fp4q_moe_mxfp4(xq["q"], xq["sf"], t, *L.dev, top_k=4, out_dtype=torch.float32)
        check(got, L, x, t, 4, True)


def test_equals_the_librarys_products():
    """One expert, one token choice of weight 1: the layer is product, activation,
    quantizer and product, bit for bit where the first product's sums agree."""
    L = Layer(3, 512, 256, 6)
    T = 20
    xq, x = tokens(T, 512, 7)
    logits = torch.full((T, 3), -float("inf"), device=DEV)
    logits[:, 1] = 0.0
    got = fq.fp4q_moe_mxfp4(xq["q"], xq["sf"], logits, *L.dev, top_k=2, out_dtype=torch.float32)
    q13, s13, q2, s2 = L.dev
    a = fq.fp4q_gemm_mxfp8_mxfp4(xq["q"], xq["sf"], q13[1].contiguous(), s13.view(3, -1)[1].contiguous())
    h = (a[:, :256].double() * torch.sigmoid(a[:, :256].double()) * a[:, 256:].double()).float()
    hq = fq.fp4q_quantize_mxfp8(h, scale_layout=fq.SCALE_SWIZZLED)
    ref = fq.fp4q_gemm_mxfp8_mxfp4(hq["q"], hq["sf"], q2[1].contiguous(), s2.view(3, -1)[1].contiguous())
    check(got, L, x, logits, 2, True)
    assert float((got - ref).norm() / ref.norm()) < 1e-2


def test_strided_output_workspace_and_empty():
    L = Layer(8, 256, 128, 8)
    xq, x = tokens(9, 256, 9)
    logits = torch.randn(9, 8, generator=torch.Generator().manual_seed(10)).to(DEV)
    big = torch.full((11, 320), 5.0, device=DEV)
    need = fq.lib().fp4q_moe_mxfp4_workspace_bytes(9, 8, 2, 256, 128)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=DEV)
    fq.fp4q_moe_mxfp4(xq["q"], xq["sf"], logits, *L.dev, top_k=2, out=big[1:10, 32:288],
                      workspace=ws[:need])
    check(big[1:10, 32:288], L, x, logits, 2, True)
    assert (ws[need:] == 0xFF).all()
    big[1:10, 32:288] = 5.0
    assert (big == 5.0).all()
    none = fq.fp4q_moe_mxfp4(xq["q"][:0], xq["sf"], logits[:0], *L.dev, top_k=2)
    assert none.shape == (0, 256)


def test_norm_router_and_layer_captured():
    """Norm with MXFP8 and y, the router's product, the layer: one decode step,
    captured in two graphs that are replayed on new inputs, and run eagerly on
    another stream in between."""
    L = Layer(16, 512, 256, 11)
    g = torch.Generator().manual_seed(12)
    w = torch.randn(512, generator=g).bfloat16().to(DEV)
    router = (torch.randn(512, 16, generator=g) * 0.1).bfloat16().to(DEV)
    args = [[(torch.randn(T, 512, generator=g)).bfloat16().to(DEV) for _ in range(2)]
            for T in (1, 24)]

    def step(x, r):
        n = fq.fp4q_rmsnorm_mxfp8(x, w, residual=r, scale_layout=fq.SCALE_SWIZZLED, want_y=True)
        logits = (n["y"].float() @ router.float())
        return n, logits, fq.fp4q_moe_mxfp4(n["q"], n["sf"], logits, *L.dev, top_k=4)

    want = [step(*a) for a in args]
    for n, logits, y in want:
        check(y, L, plain.decode8(n["q"].cpu().numpy(), n["sf"].cpu().numpy(), True), logits, 4, True)
    graphs, outs, static = [], [], [[torch.zeros_like(t) for t in a] for a in args]
    for a in static:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step(*a)[2])
        graphs.append(gr)
    for s, a in zip(static, args):
        for t, v in zip(s, a):
            t.copy_(v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for gr in graphs:
        gr.replay()
    with torch.cuda.stream(side):
        eager = [step(*a)[2] for a in args]
    torch.cuda.synchronize()
    for o, e, (_, _, ref) in zip(outs, eager, want):
        assert torch.equal(o, ref) and torch.equal(e, ref)


@pytest.mark.parametrize("T,E,k,H,I", [(20, 16, 4, 4096, 3584), (64, 24, 6, 2048, 4096),
                                       (1, 8, 8, 8192, 2048), (16, 12, 3, 4096, 2048)])
def test_large_layers(T, E, k, H, I):
    """Sizes at which the kernels take their deep rings, against FP64 products on the
    GPU of the operands as fp4q_dequantize (tested bit for bit) gives them.  Tolerance as
    above; h's moved codes are the root of a row's worst case."""
    g = torch.Generator(device=DEV).manual_seed(T)

    def w4(rows, cols):
        q = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device=DEV, generator=g)
        s = torch.randint(119, 122, (rows * cols // 32,), dtype=torch.uint8, device=DEV, generator=g)
        return q, s

    (q13, s13), (q2, s2) = w4(E * 2 * I, H), w4(E * H, I)
    xq = fq.fp4q_quantize_mxfp8(torch.randn(T, H, device=DEV, generator=g),
                                scale_layout=fq.SCALE_SWIZZLED)
    logits = torch.randn(T, E, device=DEV, generator=g)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = fq.fp4q_moe_mxfp4(xq["q"], xq["sf"], logits, q13.view(E, 2 * I, H // 2), s13,
                            q2.view(E, H, I // 2), s2, top_k=k, out_dtype=torch.float32,
                            status=status)
    assert int(status) == 0
    p = torch.from_numpy(plain.route(logits.double().cpu().numpy(), k, True)).to(DEV)

    def read(q, s, rows, cols, fmt=fq.FMT_MXFP4):
        return fq.fp4q_dequantize(fmt, q, s, rows, cols, 1, 32,
                                  scale_layout=fq.SCALE_SWIZZLED).double()

    x = read(xq["q"], xq["sf"], T, H, fq.FMT_MXFP8)
    want, mag, flip = (torch.zeros(T, H, dtype=torch.float64, device=DEV) for _ in range(3))
    for e in range(E):
        w = read(q13.view(E, -1)[e], s13.view(E, -1)[e], 2 * I, H)
        a = x @ w.t()
        h = a[:, :I] / (1 + torch.exp(-a[:, :I])) * a[:, I:]
        v, ex = plain.quantize(h.cpu().numpy())
        h = torch.from_numpy(v * np.repeat(np.ldexp(1.0, ex), 32, 1)).to(DEV)
        w = read(q2.view(E, -1)[e], s2.view(E, -1)[e], H, I)
        want += p[:, e:e + 1] * (h @ w.t())
        mag += p[:, e:e + 1] * (h.abs() @ w.abs().t())
        flip = torch.maximum(flip, p[:, e:e + 1] * h.abs().amax(1, keepdim=True) * w.abs().max())
    err = (got.double() - want).abs()
    bound = 4 * (H + I + E + 64) * 2.0 ** -22 * mag + 2 * flip * 2.0 ** -3
    assert bool((err <= bound).all())
    assert float((got.double() - want).norm() / want.norm()) < 1e-3
