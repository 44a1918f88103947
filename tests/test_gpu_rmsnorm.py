"""GPU tests of the RMS norm with MXFP8 output and of its backward pass against
the plain forms in 64 bits.

Tolerances.  A row's sum of H terms passes through at most 8 * 4 additions in a
thread, 5 in the warp and 32 across warps, 69 roundings of 2^-24 each relative
to the sum of magnitudes.  rstd halves the relative error of the mean and adds
the roundings of the division by H, the addition of eps, the root and the
reciprocal: (69 + 2) / 2 + 2 < 40 units of 2^-24.  y adds two products.  E4M3
codes are off by at most half a step (2^-4 relative, 2^-10 * 2^e below the
normal range) from the FP32 y, and a block's exponent may move by one only
where y's error moves the block maximum across a border."""
import numpy as np
import pytest
import torch

import fp4_block_scaled_04_b200 as fq
import plain_mxfp8 as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fq.lib()


def matrix(rows, cols, seed, dtype, scale=1.0, ld=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, ld or cols), generator=g) * scale
    x[:, ::37] *= 20
    return x.to(dtype).to(DEV)[:, :cols]


def f64(t):
    return t.double().cpu().numpy()


def half(dtype):
    return torch.finfo(dtype).eps / 2


def check_forward(out, s, w, eps, swizzled, y_dtype=None):
    rows, cols = s.shape
    y, rstd = plain.rmsnorm(f64(s), f64(w), eps)
    got = f64(out["rstd"])
    assert np.all(np.abs(got - rstd) <= 40 * U * rstd)
    q, sf = out["q"].cpu().numpy(), out["sf"].cpu().numpy()
    at = plain.scale_index(rows, cols // 32, swizzled)
    e = sf[at].astype(np.int64) - 127
    m = np.abs(y).reshape(rows, cols // 32, 32).max(-1)
    lo = plain.exponent((m * (1 - 2.0 ** -18)).astype(np.float32))
    hi = plain.exponent((m * (1 + 2.0 ** -18)).astype(np.float32))
    assert np.all((e >= lo) & (e <= hi))
    scale = np.repeat(np.ldexp(1.0, e), 32, 1)
    err = np.abs(plain.e4m3_values(q) * scale - y)
    bound = plain.HALF_E4M3 * np.abs(y) * (1 + 2.0 ** -18) + 2.0 ** -10 * scale + 42 * U * np.abs(y)
    assert np.all(err <= bound)
    pad = np.ones(sf.size, bool)
    pad[at.reshape(-1)] = False
    assert not sf[pad].any()
    if y_dtype is not None:
        assert np.all(np.abs(f64(out["y"]) - y) <= (half(y_dtype) * (1 + 2.0 ** -8) + 42 * U) * np.abs(y) + 1e-38)


SHAPES = [(1, 32), (1, 4096), (3, 96), (5, 512), (130, 544), (131, 1056), (9, 2080), (130, 4096),
          (7, 5120), (3, 16384), (2, 16416), (2, 32768)]


@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, FP32), (FP32, FP32), (FP32, BF16)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, dtype, wdtype):
    swizzled = (rows + cols // 32) % 2 == 0
    x, r = matrix(rows, cols, 1, dtype), matrix(rows, cols, 2, dtype)
    w = (1 + 0.2 * matrix(1, cols, 3, FP32)[0]).to(wdtype)
    layout = fq.SCALE_SWIZZLED if swizzled else fq.SCALE_LINEAR
    out = fq.fp4q_rmsnorm_mxfp8(x, w, eps=1e-5, residual=r, scale_layout=layout, want_y=True)
    s = (x.float() + r.float()).to(dtype)
    assert torch.equal(out["sum"], s)
    check_forward(out, s, w, 1e-5, swizzled, dtype)
    out = fq.fp4q_rmsnorm_mxfp8(x, w, eps=1e-5, scale_layout=layout)
    assert "sum" not in out and "y" not in out
    check_forward(out, x, w, 1e-5, swizzled)


@pytest.mark.parametrize("mode", [plain.RNE, plain.FLOOR])
def test_forward_equals_norm_then_quantize(mode):
    """FP32 y and its own quantization: the same bits as the fused output."""
    x, w = matrix(65, 1024, 4, FP32), 1 + matrix(1, 1024, 5, FP32)[0]
    for layout in (fq.SCALE_LINEAR, fq.SCALE_SWIZZLED):
        out = fq.fp4q_rmsnorm_mxfp8(x, w, e8m0_mode=mode, scale_layout=layout, want_y=True)
        ref = fq.fp4q_quantize_mxfp8(out["y"], e8m0_mode=mode, scale_layout=layout)
        assert torch.equal(out["q"], ref["q"]) and torch.equal(out["sf"], ref["sf"])


def test_zero_rows_of_values_and_eps():
    """A row of zeros: rstd = 1/sqrt(eps), codes 0; with eps 0 such a row is 0 * inf = NaN, as
    the formula says, so eps is what keeps it finite."""
    x = matrix(4, 256, 6, BF16).clone()
    x[2] = 0
    w = torch.ones(256, device=DEV)
    out = fq.fp4q_rmsnorm_mxfp8(x, w, eps=1e-6)
    assert abs(float(out["rstd"][2]) - 1e3) <= 1e3 * 40 * U
    assert not out["q"][2].any() and not out["sf"].view(4, 8)[2].any()
    check_forward(out, x, w, 1e-6, False)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("rows,cols", [(3, 96), (300, 1056)])
def test_squares_past_fp32(rows, cols, dtype):
    """A row whose squares pass FP32 has rstd 0 and normed values of 0; its
    neighbours are what they are without it."""
    x = matrix(rows, cols, 31, dtype).contiguous()
    w = matrix(1, cols, 32, BF16)[0]
    want = fq.fp4q_rmsnorm_mxfp8(x, w, want_y=True)
    x[1] = 1e25
    got = fq.fp4q_rmsnorm_mxfp8(x, w, want_y=True)
    others = [i for i in range(rows) if i != 1]
    for k in ("q", "y", "rstd"):
        assert torch.equal(got[k][others], want[k][others])
        assert not got[k][1].float().any() or k == "q"
    assert not (got["q"][1] & 0x7F).any()
    assert not got["sf"].view(rows, -1)[1].any()


@pytest.mark.parametrize("rows,cols", [(3, 96), (300, 1056)])
def test_large_weights_and_values(rows, cols):
    """Weights whose product with x would pass FP32 although y does not; a row at the
    type's largest value."""
    x = (matrix(rows, cols, 33, BF16).float() * 2.0 ** 40).to(BF16)
    w = matrix(1, cols, 34, BF16)[0].clone()
    w[5::11] = 2.0 ** 100
    check_forward(fq.fp4q_rmsnorm_mxfp8(x, w), x, w, 1e-6, False)
    x[2] = torch.finfo(BF16).max
    w[5::11] = 3.0
    out = fq.fp4q_rmsnorm_mxfp8(x, w, want_y=True)
    assert float(out["rstd"][2]) == 0 and not out["y"][2].float().any()
    keep = [i for i in range(rows) if i != 2]
    assert torch.isfinite(out["y"][keep].float()).all()


def test_strided_inputs_in_place_sum_and_empty():
    x, r = matrix(33, 640, 7, BF16, ld=704), matrix(33, 640, 8, BF16, ld=1024)
    w = matrix(1, 640, 9, BF16)[0]
    ref = fq.fp4q_rmsnorm_mxfp8(x.contiguous(), w, residual=r.contiguous())
    out = fq.fp4q_rmsnorm_mxfp8(x, w, residual=r)
    for k in ref:
        assert torch.equal(out[k], ref[k]), k
    stream = r.contiguous()
    mine = {k: torch.empty_like(v) for k, v in ref.items()}
    mine["sum"] = stream                                   # the residual stream, updated in place
    fq.fp4q_rmsnorm_mxfp8(x, w, residual=stream, out=mine)
    for k in ref:
        assert torch.equal(mine[k], ref[k]), k
    out = fq.fp4q_rmsnorm_mxfp8(x[:0], w, residual=r[:0])
    assert out["q"].shape == (0, 640) and out["sum"].shape == (0, 640)


def check_backward(got, g, s, w, rstd, d, dtype):
    G, S, W, R = f64(g), f64(s), f64(w), f64(rstd)
    D = None if d is None else f64(d)
    dx, dw = plain.rmsnorm_backward(G, S, W, R, D)
    r = R[:, None]
    # 69 roundings of the dot product, 8 of the rest; half a step of the output type
    mag = np.abs(r * W * G) + np.abs(S) * r ** 3 * np.abs(W * G * S).mean(1, keepdims=True)
    mag = mag if D is None else mag + np.abs(D)
    assert np.all(np.abs(f64(got["dx"]) - dx) <= 80 * U * mag + half(dtype) * np.abs(dx) * 1.01 + 1e-40)
    # one addition per row of the part, the parts' additions
    assert np.all(np.abs(f64(got["dweight"]) - dw) <= (S.shape[0] + 100) * U * np.abs(G * S * r).sum(0))


@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, FP32), (FP32, FP32), (FP32, BF16)])
@pytest.mark.parametrize("rows,cols", SHAPES + [(2049, 64), (700, 992)])
def test_backward(rows, cols, dtype, wdtype):
    s, g = matrix(rows, cols, 11, dtype), matrix(rows, cols, 12, dtype, 1e-2)
    d = matrix(rows, cols, 13, dtype, 1e-2)
    w = (1 + 0.2 * matrix(1, cols, 14, FP32)[0]).to(wdtype)
    rstd = fq.fp4q_rmsnorm_mxfp8(s, w)["rstd"]
    for dsum in (d, None):
        got = fq.fp4q_rmsnorm_backward(g, s, w, rstd, dsum=dsum)
        check_backward(got, g, s, w, rstd, dsum, dtype)
        again = fq.fp4q_rmsnorm_backward(g, s, w, rstd, dsum=dsum)
        assert torch.equal(got["dx"], again["dx"]) and torch.equal(got["dweight"], again["dweight"])


@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, FP32), (FP32, FP32), (FP32, BF16)])
@pytest.mark.parametrize("rows,cols", [(149, 32), (301, 512), (1190, 1024), (1185, 1056),
                                       (1184, 992), (330, 2080), (300, 4096), (599, 5120),
                                       (301, 6144), (150, 6176), (300, 8192), (149, 10240),
                                       (150, 12320)])
def test_many_rows(rows, cols, dtype, wdtype):
    """Both passes with a residual, at widths on either side of the forms' borders and
    at more rows than the GPU takes at once."""
    x, r = matrix(rows, cols, 51, dtype), matrix(rows, cols, 52, dtype)
    g = matrix(rows, cols, 53, dtype, 0.1)
    w = (1 + 0.2 * matrix(1, cols, 54, FP32)[0]).to(wdtype)
    out = fq.fp4q_rmsnorm_mxfp8(x, w, residual=r, scale_layout=fq.SCALE_SWIZZLED)
    s = (x.float() + r.float()).to(dtype)
    assert torch.equal(out["sum"], s)
    check_forward(out, s, w, 1e-6, True)
    got = fq.fp4q_rmsnorm_backward(g, s, w, out["rstd"], dsum=r)
    check_backward(got, g, s, w, out["rstd"], r, dtype)
    check_forward(fq.fp4q_rmsnorm_mxfp8(s, w), s, w, 1e-6, False)
    check_backward(fq.fp4q_rmsnorm_backward(g, s, w, out["rstd"]), g, s, w, out["rstd"], None, dtype)


def test_backward_strided_in_place_and_empty():
    s, g = matrix(50, 640, 15, BF16, ld=768), matrix(50, 640, 16, BF16, 1e-2, ld=648)
    d = matrix(50, 640, 17, BF16, 1e-2, ld=1280)
    w = matrix(1, 640, 18, BF16)[0]
    rstd = fq.fp4q_rmsnorm_mxfp8(s, w)["rstd"]
    ref = fq.fp4q_rmsnorm_backward(g.contiguous(), s.contiguous(), w, rstd, dsum=d.contiguous())
    got = fq.fp4q_rmsnorm_backward(g, s, w, rstd, dsum=d)
    assert torch.equal(got["dx"], ref["dx"]) and torch.equal(got["dweight"], ref["dweight"])
    for name in ("dy", "dsum"):
        a = {"dy": g.contiguous(), "dsum": d.contiguous()}
        out = {"dx": a[name], "dweight": torch.empty_like(ref["dweight"])}
        fq.fp4q_rmsnorm_backward(a["dy"], s, w, rstd, dsum=a["dsum"], out=out)
        assert torch.equal(out["dx"], ref["dx"]) and torch.equal(out["dweight"], ref["dweight"])
    got = fq.fp4q_rmsnorm_backward(g[:0], s[:0], w, rstd[:0])
    assert got["dx"].shape == (0, 640) and not got["dweight"].any()


def test_gradient_against_differences():
    """Central differences of the plain forward pass in 64 bits, for loss =
    sum(y g) + sum(s d): error h^2 / 6 times the third derivative (about 1e-8
    here) next to FP32 rounding of the kernel."""
    rng = np.random.default_rng(3)
    s, g, d = (rng.standard_normal((3, 64)).astype(np.float32) for _ in range(3))
    w = rng.standard_normal(64).astype(np.float32)
    t = [torch.from_numpy(a).to(DEV) for a in (s, g, d, w)]
    rstd = fq.fp4q_rmsnorm_mxfp8(t[0], t[3], eps=1e-5)["rstd"]
    got = fq.fp4q_rmsnorm_backward(t[1], t[0], t[3], rstd, dsum=t[2])

    def loss(s_, w_):
        return float((plain.rmsnorm(s_, w_, 1e-5)[0] * g).sum() + (s_ * d).sum())

    S, W, h = s.astype(np.float64), w.astype(np.float64), 1e-4
    for i in rng.choice(3 * 64, 24, replace=False):
        e = np.zeros(3 * 64)
        e[i] = h
        e = e.reshape(3, 64)
        num = (loss(S + e, W) - loss(S - e, W)) / (2 * h)
        assert abs(num - float(got["dx"].view(-1)[i])) <= 1e-5 * (1 + abs(num))
    for i in range(0, 64, 5):
        e = np.zeros(64)
        e[i] = h
        num = (loss(S, W + e) - loss(S, W - e)) / (2 * h)
        assert abs(num - float(got["dweight"][i])) <= 1e-5 * (1 + abs(num))


def test_captured_passes_share_no_state():
    """Forward and backward captured into two graphs, replayed on new inputs
    while eager calls of the same shapes run in between."""
    w = matrix(1, 1024, 20, BF16)[0]
    args = [[matrix(300, 1024, 30 + 4 * i + j, BF16) for j in range(4)] for i in range(2)]

    def step(x, r, g, d):
        o = fq.fp4q_rmsnorm_mxfp8(x, w, residual=r, scale_layout=fq.SCALE_SWIZZLED)
        return {**o, **fq.fp4q_rmsnorm_backward(g, o["sum"], w, o["rstd"], dsum=d)}

    want = [step(*a) for a in args]
    step(*args[0])
    graphs, outs = [], []
    static = [[torch.zeros_like(t) for t in a] for a in args]
    for a in static:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step(*a))
        graphs.append(gr)
    for s_, a in zip(static, args):
        for t, v in zip(s_, a):
            t.copy_(v)
    for gr in graphs:
        gr.replay()
    eager = step(*args[0])
    torch.cuda.synchronize()
    for o, ref in zip(outs + [eager], want + [want[0]]):
        for k in ref:
            assert torch.equal(o[k], ref[k]), k
