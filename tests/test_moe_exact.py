"""The mixture-of-experts layer on operands whose inner steps are exact, so that nothing
but the routing weights and the last sums rounds.

The first product adds small whole numbers (exact in any order).  Each gate row has one
large weight on x's first value, +-768 in all, beside which the rest stays below 500: a
gate is at least 18, where FP32's silu(g) = g / (1 + exp(-g)) is g, or at most -110, where
it is -0.  So h = silu(g) u is a whole number below 2^24 and its MXFP8 code is fixed: no
code may move.

Tolerance.  Logits are BF16 values, whose differences are exact in FP32.  exp is within 2
units in the last place (4 units of 2^-24), the softmax's sum adds at most 13 roundings to
that, the division one: 22.  Renormalizing divides by the sum of such numbers: below 50.
The weighted sum takes at most 16 multiply-adds and 8 additions.  With one weight to a row
of W2 the second product is exact: 80 units of 2^-24 of sum p |h W2| in all.  With dense
weights its additions come on top, 2^-22 each as for the plain product: (I + 2) 2^-22 of
sum p |h| |W2|.  BF16 outputs add half a step."""
import numpy as np
import pytest
import torch

import fp4_block_scaled_04_b200 as fq
import plain_mxfp8 as plain

DEV = "cuda"
U = 2.0 ** -24
E4M3 = {v: (0x80 if v < 0 else 0) | c for v, c in [(0, 0), (1, 0x38), (2, 0x40), (16, 0x58)]}
E4M3.update({-1: 0xB8, -2: 0xC0})


def pack(code):
    return code[..., 0::2] | code[..., 1::2] << 4


def swizzle(byte):
    out = np.zeros(-(-byte.shape[0] // 128) * 128 * byte.shape[1], np.uint8)
    out[plain.scale_index(*byte.shape, True)] = byte
    return out


class Case:
    def __init__(self, T, E, k, H, I, dense, seed):
        rng = np.random.default_rng(seed)
        self.shape = T, E, k, H, I
        self.dense = dense
        # x: -2..2, its first value 16
        x = rng.integers(-2, 3, (T, H))
        x[:, 0] = 16
        x[:, 1:32] = 0                              # the block of the large weight
        self.x = x.astype(np.float64)
        self.xq = np.vectorize(E4M3.get)(x).astype(np.uint8)
        self.xsf = swizzle(np.full((T, H // 32), 127, np.uint8))
        # W13: -1, 0, 1, few of them on wide rows; gate rows +-48 = 6 * 2^3 in front
        few = min(0.5, 128 / H)
        sign = rng.random((E, 2 * I, H)) < 0.5
        code = (2 * (rng.random((E, 2 * I, H)) < few)).astype(np.uint8)
        code |= (sign & (code > 0)).astype(np.uint8) << 3
        code[:, :, :32] = 0
        code[:, :I, 0] = np.where(rng.random((E, I)) < 0.5, 7, 15)
        byte = np.full((E, 2 * I, H // 32), 127, np.uint8)
        byte[:, :I, 0] = 130
        self.q13, self.s13 = pack(code), swizzle(byte.reshape(E * 2 * I, H // 32))
        # W2: one weight a row, or all of them
        if dense:
            code = rng.integers(0, 16, (E, H, I)).astype(np.uint8)
        else:
            code = np.zeros((E, H, I), np.uint8)
            at = rng.integers(0, I, (E, H))
            np.put_along_axis(code, at[..., None], (rng.integers(1, 8, (E, H)) |
                                                    rng.integers(0, 2, (E, H)) << 3
                                                    ).astype(np.uint8)[..., None], 2)
        self.q2 = pack(code)
        self.s2 = swizzle(rng.integers(125, 130, (E * H, I // 32)).astype(np.uint8))
        self.logits = torch.from_numpy(rng.standard_normal((T, E)) * 1.5).bfloat16()

    def want(self, renormalize, weight=None):
        """Output, and the sum of magnitudes that its tolerance is relative to.  weight:
        an array that the routing weights are multiplied with (a planted mistake)."""
        T, E, k, H, I = self.shape
        p = plain.route(self.logits.double().numpy(), k, renormalize)
        if weight is not None:
            p = p * weight
        out, mag = np.zeros((T, H)), np.zeros((T, H))
        for e in np.nonzero(p.any(0))[0]:
            w = plain.decode4(self.q13[e], self.s13.reshape(E, -1)[e])
            a = self.x @ w.T
            g, u = a[:, :I], a[:, I:]
            assert np.all((g >= 18) | (g <= -110)) and np.abs(g * u).max() < 2 ** 24
            v, ex = plain.quantize(np.where(g > 0, g * u, 0.0))
            h = v * np.repeat(np.ldexp(1.0, ex), 32, 1)
            w = plain.decode4(self.q2[e], self.s2.reshape(E, -1)[e])
            out += p[:, e:e + 1] * (h @ w.T)
            mag += p[:, e:e + 1] * (np.abs(h) @ np.abs(w).T)
        return out, mag

    def within(self, got, out, mag, dtype):
        I = self.shape[4]
        rel = 80 * U + ((I + 2) * 2.0 ** -22 if self.dense else 0.0)
        half = 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2
        return np.abs(got - out) <= rel * (1 + half) * mag + half * np.abs(out) + 1e-30


CASES = [  # T, E, k, H, I: both sides of 16, 32 and 64 tokens, few and many experts
    (1, 1, 1, 128, 128), (1, 8, 2, 256, 128), (1, 64, 8, 1024, 512), (2, 5, 3, 384, 256),
    (13, 8, 2, 2048, 1024), (16, 2, 2, 128, 640), (17, 40, 6, 512, 384), (31, 256, 16, 256, 128),
    (32, 8, 8, 1024, 256), (33, 12, 1, 640, 256), (64, 16, 4, 512, 512), (64, 4, 4, 1152, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("renormalize,dtype", [(True, torch.bfloat16), (False, torch.float32),
                                               (True, torch.float32)])
@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("T,E,k,H,I", CASES)
def test_layer_on_exact_operands(T, E, k, H, I, dense, renormalize, dtype):
    c = Case(T, E, k, H, I, dense, T + E)
    dev = [torch.from_numpy(a).to(DEV) for a in (c.xq, c.xsf, c.q13, c.s13, c.q2, c.s2)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, mag = c.want(renormalize)
    for logits in (c.logits.to(DEV), c.logits.float().to(DEV)):
        got = fq.fp4q_moe_mxfp4(*dev[:2], logits, *dev[2:], top_k=k, renormalize=renormalize,
                                out_dtype=dtype, status=status)
        assert int(status) == 0
        ok = c.within(got.double().cpu().numpy(), out, mag, dtype)
        assert ok.all(), np.argwhere(~ok)[:5]


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 16, 20, 64])
def test_one_expert_of_weight_one_is_exact(T):
    """One choice left by the mask: its weight is 1 and the output the library's own
    products around h, bit for bit."""
    E, H, I = 3, 512, 256
    c = Case(T, E, 2, H, I, False, 7)
    c.logits[:] = -float("inf")
    c.logits[torch.arange(T), torch.arange(T) % E] = 0.5
    xq, xsf, q13, s13, q2, s2 = [torch.from_numpy(a).to(DEV)
                                 for a in (c.xq, c.xsf, c.q13, c.s13, c.q2, c.s2)]
    got = fq.fp4q_moe_mxfp4(xq, xsf, c.logits.to(DEV), q13, s13, q2, s2, top_k=2,
                            out_dtype=torch.float32)
    for e in range(E):
        t = torch.arange(T) % E == e
        a = fq.fp4q_gemm_mxfp8_mxfp4(xq, xsf, q13[e], s13.view(E, -1)[e])
        h = torch.where(a[:, :I] > 0, a[:, :I], 0.0) * a[:, I:]
        hq = fq.fp4q_quantize_mxfp8(h, scale_layout=fq.SCALE_SWIZZLED)
        ref = fq.fp4q_gemm_mxfp8_mxfp4(hq["q"], hq["sf"], q2[e], s2.view(E, -1)[e])
        assert torch.equal(got[t], ref[t])
    assert np.array_equal(got.double().cpu().numpy(), c.want(True)[0])


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 256, 128), (2, 5, 3, 384, 256),
                                       (17, 40, 6, 512, 384), (64, 4, 4, 1152, 128)])
def test_tolerance_catches_mistakes(T, E, k, H, I, dense, renormalize):
    """On the CPU: every third token's weights by 1.05, each token's largest by 1.01, or a
    token's smallest expert left out, is outside the tolerance (in BF16 too, but for the
    second, which is about half a step)."""
    c = Case(T, E, k, H, I, dense, T + E)
    out, mag = c.want(renormalize)
    p = plain.route(c.logits.double().numpy(), k, renormalize)
    some = np.arange(T) % 3 == 0
    scaled, one, dropped = np.ones((T, E)), np.ones((T, E)), np.ones((T, E))
    scaled[some] = 1.05
    one[np.arange(T), p.argmax(1)] = 1.01
    dropped[0, np.argmin(np.where(p[0] > 0, p[0], 2))] = 0
    assert c.within(out, out, mag, torch.float32).all()
    for mistake, dtypes in ((scaled, (torch.float32, torch.bfloat16)), (one, (torch.float32,)),
                            (dropped, (torch.float32, torch.bfloat16))):
        bad = c.want(renormalize, mistake)[0]
        for dt in dtypes:
            got = torch.from_numpy(bad).to(dt).double().numpy()
            rows = ~c.within(got, out, mag, dt).all(1)
            assert np.array_equal(rows, (p * (mistake != 1)).any(1))
