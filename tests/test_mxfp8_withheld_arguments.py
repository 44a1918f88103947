"""Refusals of the test hooks that make a wait run out, on the CPU."""
import ctypes

import pytest

import fp4_block_scaled_04_b200 as fq
from fp4_block_scaled_04_b200 import build

A = ctypes.c_void_p(0x7F0000000000)                # 16-byte aligned, never dereferenced
OK, ARG, SHAPE, ALIGN, WS = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    build.build()
    return fq.lib()


def test_withheld_loads_of_the_product(L):
    def call(K=256, loads=(0, 0), status=A, M=3, ldc=128):
        return L.fp4q_gemm_mxfp8_mxfp4_withhold_loads(A, A, A, A, M, 128, K, A, 0, ldc, *loads,
                                                      status, None)
    assert call(K=0) == ARG and call(status=None) == ARG
    assert call(loads=(-1, 0)) == ARG and call(loads=(0, -1)) == ARG
    assert call(K=160) == SHAPE and call(ldc=120) == ARG and call(ldc=129) == ALIGN
    assert call(M=0) == OK


def test_withheld_loads_of_the_expert_layer(L):
    def call(T=5, product=1, loads=(0, 0), status=A, n=1 << 30, H=256):
        return L.fp4q_moe_mxfp4_withhold_loads(A, A, A, 1, A, A, A, A, T, 8, 2, H, 128, 1, A, 0,
                                               256, A, n, product, *loads, status, None)
    assert call(product=0) == ARG and call(product=3) == ARG and call(status=None) == ARG
    assert call(loads=(-1, 0)) == ARG and call(loads=(0, -1)) == ARG
    assert call(T=65) == SHAPE and call(H=192) == SHAPE and call(n=0) == WS
    assert call(T=0) == OK
