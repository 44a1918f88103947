"""Plain 64-bit forms of the MXFP8 operators for the tests (numpy, from the
definitions in include/fp4q.h; no code of the library or of the oracle)."""
import numpy as np

RNE, CEIL, FLOOR = 0, 1, 2
HALF_E4M3 = 2.0 ** -4                              # half a step, relative


def exponent(m, mode=CEIL):
    """Unbiased E8M0 exponent of blocks with maximum m (float32 values)."""
    m = np.asarray(m, np.float32)
    if mode == FLOOR:
        _, e = np.frexp(m.astype(np.float64))
        e = e - 1 - 8
        zero = m == 0
    else:
        t = (m / np.float32(448)).astype(np.float64)   # one FP32 rounding
        f, e = np.frexp(t)                             # t = f 2^e, f in [.5, 1)
        if mode == CEIL:
            e = np.where(f > 0.5, e, e - 1)
        else:                                          # nearest, ties to the even biased exponent
            low = e - 1
            e = np.where(f > 0.75, e, np.where(f < 0.75, low,
                                               np.where((low + 127) % 2 == 0, low, e)))
        zero = t == 0
    return np.where(zero, -127, np.clip(e, -127, 127)).astype(np.int64)


def e4m3_round(v):
    """Nearest E4M3 value, ties to even, saturating at 448."""
    v = np.asarray(v, np.float64)
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.clip(np.round(v / step) * step, -448, 448)


def e4m3_values(code):
    c = np.asarray(code, np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, np.ldexp(8 + m, e - 10))
    return np.where(c >= 128, -v, v)


def quantize(x, mode=CEIL):
    """Float64 [R, C] holding FP32 values -> (code values [R, C], exponents [R, C/32])."""
    R, C = x.shape
    b = x.reshape(R, C // 32, 32)
    e = exponent(np.abs(b).max(-1), mode)
    v = np.ldexp(b, -e[..., None])
    v = v.astype(np.float32).astype(np.float64)        # RN(x 2^-e)
    return e4m3_round(v).reshape(R, C), e


def scale_index(rows, scols, swizzled):
    r, c = np.arange(rows)[:, None], np.arange(scols)[None, :]
    if not swizzled:
        return r * scols + c
    return ((r // 128) * (-(-scols // 4)) + c // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + c % 4


def decode8(q, sf, swizzled):
    R, C = q.shape
    e = np.asarray(sf).reshape(-1)[scale_index(R, C // 32, swizzled)].astype(np.int64) - 127
    return e4m3_values(q) * np.repeat(np.ldexp(1.0, e), 32, 1)


def decode4(q, sf, swizzled=True):
    """Packed E2M1 codes [R, C/2] and E8M0 bytes -> float64 [R, C]."""
    q = np.asarray(q, np.uint8)
    R, C = q.shape[0], 2 * q.shape[1]
    grid = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    code = np.empty((R, C), np.int64)
    code[:, 0::2], code[:, 1::2] = q & 15, q >> 4
    e = np.asarray(sf).reshape(-1)[scale_index(R, C // 32, swizzled)].astype(np.int64) - 127
    return np.where(code >= 8, -1, 1) * grid[code & 7] * np.repeat(np.ldexp(1.0, e), 32, 1)


def rmsnorm(s, w, eps):
    """(y, rstd) in float64 of rows s."""
    rstd = 1 / np.sqrt((s * s).mean(1) + eps)
    return s * rstd[:, None] * w, rstd


def rmsnorm_backward(g, s, w, rstd, d=None):
    r = rstd[:, None]
    dx = r * (w * g - s * r * r * (w * g * s).mean(1, keepdims=True))
    return (dx if d is None else dx + d), (g * s * r).sum(0)


def route(logits, k, renormalize):
    """[T, E] weights (0 where an expert is not chosen) in float64."""
    p = np.zeros(logits.shape)
    for t, row in enumerate(np.asarray(logits, np.float64)):
        row = np.where(np.isnan(row), -np.inf, row)
        if row.max() == -np.inf:
            continue
        q = np.exp(row - row.max())
        q /= q.sum()
        at = [e for e in np.argsort(-row, kind="stable")[:k] if q[e] > 0]
        p[t, at] = q[at] / (q[at].sum() if renormalize else 1.0)
    return p


def moe(x, p, w13, w2):
    """Output [T, H], and the bound of a difference that comes from h's codes
    moving by one step: the sum over one code of p 2^-3 |h| |W2|, at its
    largest.  x [T, H], p [T, E] float64; w13(e), w2(e) give the weights."""
    T, H = x.shape
    out, mag, flip = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    for e in np.nonzero(p.any(0))[0]:
        a = x @ w13(e).T
        I = a.shape[1] // 2
        with np.errstate(over="ignore"):
            h = a[:, :I] / (1 + np.exp(-a[:, :I])) * a[:, I:]
        v, ex = quantize(h)
        hq = v * np.repeat(np.ldexp(1.0, ex), 32, 1)
        W = w2(e)
        out += p[:, e:e + 1] * (hq @ W.T)
        mag += p[:, e:e + 1] * (np.abs(hq) @ np.abs(W).T)
        flip = np.maximum(flip, p[:, e:e + 1] * np.abs(hq).max(1, keepdims=True) * np.abs(W).max())
    return out, mag, flip * 2.0 ** -3
