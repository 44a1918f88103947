"""GPU tests of the norm's roundings where every sum is exact: small whole numbers, whose
squares and products add up without rounding in any order.

What is left: mean + eps is rounded once (2^-24 relative), which the root halves, and the
root is within half a step (2^-24) but for terms far below it: (1/2 + 1) 2^-24 for rstd.
The backward pass's mean is rounded once, and so is its product with rstd = 1 and x = 1.
The bounds get 2^-10 of themselves on top for the terms of second order."""
import pytest
import torch

import fp4_block_scaled_04_b200 as fq

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
# both sides of the forms' borders; no powers of two, for which 1 / cols is exact, but one
COLS = [96, 544, 1056, 1504, 2080, 3488, 4096, 5120, 7264, 10240, 16416]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fq.lib()


def whole(rows, cols, seed, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randint(-7, 8, (rows, cols), device=DEV, generator=g)
    # rows of many magnitudes of the mean
    keep = torch.rand(rows, 1, device=DEV, generator=g) ** 2
    x *= torch.rand(rows, cols, device=DEV, generator=g) < keep
    x[:, 0] = 1
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [147, 3000])
@pytest.mark.parametrize("cols", COLS)
def test_rstd(rows, cols, dtype):
    x = whole(rows, cols, cols, dtype)
    w = torch.ones(cols, device=DEV)
    for eps in (0.0, 2.0 ** -10):
        got = fq.fp4q_rmsnorm_mxfp8(x, w, eps=eps)["rstd"].double()
        want = 1 / torch.sqrt(x.double().square().sum(1) / cols + eps)
        err = ((got - want) / want).abs().max()
        assert float(err) <= 1.5 * U * (1 + 2.0 ** -10), float(err) / U


@pytest.mark.parametrize("rows", [147, 3000])
@pytest.mark.parametrize("cols", COLS)
def test_mean_of_the_backward_pass(rows, cols):
    """With rstd = 1, x = 1 and no gradient of its own a column's dx is minus the mean
    of w g x."""
    x = whole(rows, cols, cols + 1, torch.float32)
    g = whole(rows, cols, cols + 2, torch.float32)
    g[:, 0] = 0
    g[:, 1] = 5
    x[:, 1] = 3
    w = torch.ones(cols, device=DEV)
    got = fq.fp4q_rmsnorm_backward(g, x, w, torch.ones(rows, device=DEV))["dx"][:, 0].double()
    want = -(g.double() * x.double()).sum(1) / cols
    assert bool(((got - want).abs() <= U * (1 + 2.0 ** -10) * want.abs()).all())
