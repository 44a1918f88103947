"""GPU test of the MXFP8 operators as a model runs them: a stack of layers, each the
norm with the residual stream, the product, the quantizer, a second product back into the
stream, the norm and the expert layer, with kernels of other libraries in between.  The
kernels of this path may begin while their predecessor drains, so a stack that is launched
without a pause, many times over the same buffers, has to give the bits of one in which
every call is waited for."""
import pytest
import torch

import fp4_block_scaled_04_b200 as fq

pytestmark = pytest.mark.gpu
DEV = "cuda"
SW = fq.SCALE_SWIZZLED


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fq.lib()


class Stack:
    def __init__(self, layers, H, I, E):
        g = torch.Generator(device=DEV).manual_seed(1)

        def w4(rows, cols):
            w = torch.randn(rows, cols, device=DEV, generator=g) / cols ** 0.5
            o = fq.fp4q_quantize_mxfp4(w, scale_layout=SW)
            return o["q_row"], o["sf_row"]

        self.H, self.I, self.E = H, I, E
        self.layers = []
        for _ in range(layers):
            q13, s13 = w4(E * 2 * I, H)
            q2, s2 = w4(E * H, I)
            self.layers.append(dict(
                g1=torch.rand(H, device=DEV, generator=g) + 0.5,
                g2=torch.rand(H, device=DEV, generator=g).bfloat16() + 0.5,
                up=w4(2 * H, H), down=w4(H, 2 * H),
                router=torch.randn(H, E, device=DEV, generator=g).bfloat16(),
                experts=(q13.view(E, 2 * I, H // 2), s13, q2.view(E, H, I // 2), s2)))

    def __call__(self, x, pause=False, bufs=None):
        """x [T, H] BF16 -> the stream after all layers and every call's outputs."""
        made = []

        def did(v):
            made.append(v)
            if pause:
                torch.cuda.synchronize()
            return v

        def buf(like):
            return None if bufs is None else bufs[len(made)]

        stream, delta = torch.zeros_like(x), x
        for l in self.layers:
            n = did(fq.fp4q_rmsnorm_mxfp8(delta, l["g1"], residual=stream, scale_layout=SW,
                                          out=buf(0)))
            a = did(fq.fp4q_gemm_mxfp8_mxfp4(n["q"], n["sf"], *l["up"], out_dtype=torch.bfloat16,
                                             out=buf(0)))
            q = did(fq.fp4q_quantize_mxfp8(a, scale_layout=SW, out=buf(0)))
            y = did(fq.fp4q_gemm_mxfp8_mxfp4(q["q"], q["sf"], *l["down"],
                                             out_dtype=torch.bfloat16, out=buf(0)))
            n = did(fq.fp4q_rmsnorm_mxfp8(y, l["g2"], residual=n["sum"], scale_layout=SW,
                                          want_y=True, out=buf(0)))
            stream = n["sum"]
            if x.shape[0] <= 64:
                logits = n["y"] @ l["router"]
                delta = did(fq.fp4q_moe_mxfp4(n["q"], n["sf"], logits.float(), *l["experts"],
                                              top_k=2, out=buf(0)))
            else:
                delta = n["y"]
        return made


def bits(made):
    return [t.clone() for v in made for t in (v.values() if isinstance(v, dict) else [v])]


@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_a_stack_without_a_pause(T):
    stack = Stack(4, 512, 256, 8)
    x = torch.randn(T, 512, device=DEV, generator=torch.Generator(device=DEV).manual_seed(T)
                    ).bfloat16()
    made = stack(x, pause=True)
    want = bits(made)
    for v in want:
        if v.is_floating_point():
            assert torch.isfinite(v).all()
    for _ in range(20):                                 # the same buffers again and again
        made = stack(x, bufs=made)
    for a, b in zip(bits(made), want):
        assert torch.equal(a, b)
    # the same without a pause in a graph, replayed back to back
    static, g = x.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = stack(static)
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(bits(out), want):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    """Two stacks of different sizes on two streams at the same time."""
    stack = Stack(2, 1024, 256, 16)
    xs = [torch.randn(T, 1024, device=DEV, generator=torch.Generator(device=DEV).manual_seed(T)
                      ).bfloat16() for T in (7, 64)]
    want = [bits(stack(x, pause=True)) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    got = [None, None]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for i, (s, x) in enumerate(zip(streams, xs)):
            with torch.cuda.stream(s):
                got[i] = stack(x)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(bits(g), w):
            assert torch.equal(a, b)


def test_training_step_gradients_of_a_layer():
    """norm -> product, backward through both: the gradients that a training step takes
    equal the formulas on the library's own operands (the quantizers pass theirs through)."""
    g = torch.Generator(device=DEV).manual_seed(5)
    T, H, N = 200, 512, 384
    x, r = (torch.randn(T, H, device=DEV, generator=g).bfloat16() for _ in range(2))
    gamma = torch.rand(H, device=DEV, generator=g) + 0.5
    w = (torch.randn(N, H, device=DEV, generator=g) / H ** 0.5).bfloat16()
    qw = fq.fp4q_quantize_mxfp4(w, layouts=fq.ROWWISE | fq.COLWISE, scale_layout=SW)
    n = fq.fp4q_rmsnorm_mxfp8(x, gamma, residual=r, scale_layout=SW)
    dc = (torch.randn(T, N, device=DEV, generator=g) * 1e-2).bfloat16()
    q = fq.fp4q_quantize_mxfp8(dc, scale_layout=SW)
    dy = fq.fp4q_gemm_mxfp8_mxfp4(q["q"], q["sf"], qw["q_col"], qw["sf_col"],
                                  out_dtype=torch.bfloat16)
    got = fq.fp4q_rmsnorm_backward(dy, n["sum"], gamma, n["rstd"], dsum=x)
    s = n["sum"].double().requires_grad_()
    gam = gamma.double().requires_grad_()
    y = s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-6) * gam
    (y * dy.double()).sum().add((s * x.double()).sum()).backward()
    half = torch.finfo(torch.bfloat16).eps / 2
    err = (got["dx"].double() - s.grad).abs()
    assert bool((err <= half * 1.01 * s.grad.abs() + 80 * 2.0 ** -24 * s.grad.abs().max()).all())
    err = (got["dweight"].double() - gam.grad).abs()
    assert bool((err <= 300 * 2.0 ** -24 * (dy.double() * y.detach() / gamma).abs().sum(0)).all())
