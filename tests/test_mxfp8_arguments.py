"""Refusals of the MXFP8 calls, on the CPU: bad arguments are rejected on the
host with the documented status before a device is touched."""
import ctypes

import pytest

import fp4_block_scaled_04_b200 as fq
from fp4_block_scaled_04_b200 import build

A = ctypes.c_void_p(0x7F0000000000)                # 16-byte aligned, never dereferenced
A2 = ctypes.c_void_p(0x7F1000000000)
ODD = ctypes.c_void_p(0x7F0000000008)
OK, ARG, SHAPE, ALIGN, WS = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    build.build()
    return fq.lib()


def quantize(L, x=A, dtype=0, rows=5, cols=64, ld=64, mode=1, q=A, sf=A, layout=0):
    return L.fp4q_quantize_mxfp8(x, dtype, rows, cols, ld, mode, q, sf, layout, None)


def test_quantize(L):
    assert quantize(L, dtype=2) == ARG and quantize(L, ld=32) == ARG
    assert quantize(L, mode=3) == ARG and quantize(L, layout=2) == ARG
    assert quantize(L, rows=-1) == ARG and quantize(L, x=None) == ARG
    assert quantize(L, q=None) == ARG and quantize(L, sf=None) == ARG
    assert quantize(L, cols=48) == SHAPE
    assert quantize(L, x=ODD) == ALIGN and quantize(L, q=ODD) == ALIGN
    assert quantize(L, ld=65) == ALIGN
    assert quantize(L, rows=0, x=None, q=None, sf=None) == OK
    assert L.fp4q_dequantize(7, A, A, 0, 1, 32, None, 5, 48, A, 1, None) == SHAPE
    assert L.fp4q_dequantize(8, A, A, 0, 1, 32, None, 5, 64, A, 1, None) == ARG


def norm(L, x=A, dtype=0, rows=5, cols=64, ld=64, res=A2, ld_res=64, w=A, wdtype=0, eps=1e-6,
         mode=1, q=A, sf=A, layout=0, rstd=A, s=None, y=None):
    return L.fp4q_rmsnorm_mxfp8(x, dtype, rows, cols, ld, res, ld_res, w, wdtype, eps, mode, q,
                                sf, layout, rstd, s, y, None)


def test_norm(L):
    assert norm(L, dtype=2) == ARG and norm(L, wdtype=2) == ARG and norm(L, ld_res=32) == ARG
    assert norm(L, eps=-1.0) == ARG and norm(L, eps=float("nan")) == ARG
    assert norm(L, mode=3) == ARG and norm(L, layout=2) == ARG
    assert norm(L, w=None) == ARG and norm(L, q=None) == ARG and norm(L, sf=None) == ARG
    assert norm(L, cols=48) == SHAPE
    assert norm(L, cols=32800, ld=32800, ld_res=32800) == SHAPE
    for k in ("x", "res", "w", "q", "rstd", "s", "y"):
        assert norm(L, **{k: ODD}) == ALIGN
    assert norm(L, s=A, ld=128) == ARG                 # in place, but not at the same places
    assert norm(L, s=A2, ld_res=128) == ARG
    assert norm(L, y=A) == ARG and norm(L, y=A2) == ARG
    assert norm(L, s=ctypes.c_void_p(0x7F2000000000), y=ctypes.c_void_p(0x7F2000000000)) == ARG
    assert norm(L, rows=0) == OK


def backward(L, dy=A, ld_dy=64, x=A2, ld=64, dtype=0, w=A, wdtype=0, rstd=A, dsum=None,
             ld_dsum=64, rows=5, cols=64, dx=A, dw=A, ws=A, n=1 << 20):
    return L.fp4q_rmsnorm_backward(dy, ld_dy, x, ld, dtype, w, wdtype, rstd, dsum, ld_dsum, rows,
                                   cols, dx, dw, ws, n, None)


def test_norm_backward(L):
    assert backward(L, dtype=2) == ARG and backward(L, wdtype=2) == ARG
    assert backward(L, ld_dy=32) == ARG and backward(L, dsum=A, ld_dsum=32) == ARG
    for k in ("dy", "x", "w", "rstd", "dx", "dw"):
        assert backward(L, **{k: None}) == ARG
    assert backward(L, cols=48) == SHAPE
    assert backward(L, ld_dy=32800, ld=32800, cols=32800) == SHAPE
    need = L.fp4q_rmsnorm_backward_workspace_bytes(5, 64)
    assert need == 5 * 64 * 4 and L.fp4q_rmsnorm_backward_workspace_bytes(0, 64) == 0
    assert backward(L, n=need - 1) == WS and backward(L, ws=None) == WS
    for k in ("dy", "x", "w", "rstd", "dsum", "dx", "dw", "ws"):
        assert backward(L, **{k: ODD}) == ALIGN
    assert backward(L, dx=A2) == ARG                   # dx may not be x
    assert backward(L, ld_dy=128) == ARG               # in place, but not at the same places


def gemm(L, qa=A, sfa=A, qb=A, sfb=A, M=3, N=128, K=256, c=A, dtype=0, ldc=128, status=None):
    return L.fp4q_gemm_mxfp8_mxfp4(qa, sfa, qb, sfb, M, N, K, c, dtype, ldc, status, None)


def test_gemm(L):
    assert gemm(L, dtype=2) == ARG and gemm(L, ldc=120) == ARG and gemm(L, M=-1) == ARG
    for k in ("qa", "sfa", "qb", "sfb", "c"):
        assert gemm(L, **{k: None}) == ARG and gemm(L, **{k: ODD}) == ALIGN
    assert gemm(L, qb=ctypes.c_void_p(0x7F0000000010)) == ALIGN     # 32 bytes for the weights
    assert gemm(L, N=64, ldc=64) == SHAPE and gemm(L, K=160) == SHAPE
    assert gemm(L, M=1 << 20, N=1 << 29, ldc=1 << 29) == SHAPE
    assert gemm(L, ldc=129) == ALIGN
    assert gemm(L, M=0, qa=None, c=None) == OK and gemm(L, N=0, ldc=0) == OK


def moe(L, xq=A, xsf=A, logits=A, ldt=1, w13=A, sf13=A, w2=A, sf2=A, T=5, E=8, k=2, H=256, I=128,
        renorm=1, out=A, dtype=0, ldo=256, ws=A, n=1 << 30, status=None):
    return L.fp4q_moe_mxfp4(xq, xsf, logits, ldt, w13, sf13, w2, sf2, T, E, k, H, I, renorm, out,
                            dtype, ldo, ws, n, status, None)


def test_moe(L):
    assert moe(L, ldt=2) == ARG and moe(L, dtype=2) == ARG and moe(L, ldo=248) == ARG
    assert moe(L, T=-1) == ARG and moe(L, E=0) == ARG and moe(L, k=0) == ARG and moe(L, k=9) == ARG
    assert moe(L, T=65) == SHAPE and moe(L, E=257) == SHAPE and moe(L, E=64, k=17) == SHAPE
    assert moe(L, H=192) == SHAPE and moe(L, I=96) == SHAPE and moe(L, I=0) == SHAPE
    for p in ("xq", "xsf", "logits", "w13", "sf13", "w2", "sf2", "out"):
        assert moe(L, **{p: None}) == ARG and moe(L, **{p: ODD}) == ALIGN
    assert moe(L, w2=ctypes.c_void_p(0x7F0000000010)) == ALIGN      # 32 bytes for the weights
    assert moe(L, ws=ctypes.c_void_p(0x7F0000000080)) == ALIGN      # 256 for the workspace
    need = L.fp4q_moe_mxfp4_workspace_bytes(5, 8, 2, 256, 128)
    assert need > 5 * 2 * 128 and L.fp4q_moe_mxfp4_workspace_bytes(0, 8, 2, 256, 128) == 0
    assert moe(L, n=need - 1) == WS and moe(L, ws=None) == WS
    assert moe(L, T=0, xq=None, out=None, ws=None) == OK
