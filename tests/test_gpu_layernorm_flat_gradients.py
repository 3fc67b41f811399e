"""Layer norm backward where the gradient's mean cancels it: in a constant row
h = 0 and rstd = 1 / sqrt(eps) = 10^6, so dx = rstd (t - mean(t)), and with the
same t in the whole row dx is 0.  Where t's significand (8 or 11 bits) times
the number of columns is below 2^24, every partial sum is exact, so the mean is,
and so is the zero.  Elsewhere, and where a gradient has only a few ulps around
its mean, the roundings of the mean are what is left: u = 2^-24 and a chain of
k = 80 + cols / 256 additions leave it within (k + 2) u max|t|, and dx within rstd
times that and its own roundings."""
import math
import pytest
import torch

from gradient_reduce_optimizer_gb300 import build as gbuild
from gradient_reduce_optimizer_gb300 import capi

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()


def backward(dy, x, weight, mean, rstd):
    rows, cols = x.shape
    dx = torch.empty(rows, cols, device=DEV, dtype=x.dtype)
    capi.cc_layernorm_backward(dy, x, weight, mean, rstd, dx, None, None, rows, cols)
    return dx


# rows in vectors of one warp and several, read twice, of odd lengths, strided
COLS = [41, 47, 96, 600, 1000, 1001, 1023, 3000, 5001, 8200, 16383, 16384]


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("cols", COLS)
def test_the_same_gradient_in_the_whole_row(cols, dtype, strided):
    values = torch.tensor([1.0, 3.0, -0.1, 7.3, 1e-3, -1 / 3], device=DEV).to(dtype)
    rows = len(values)
    pad = 3 if strided else 0
    x = torch.full((rows, cols + pad), 2.0, device=DEV, dtype=dtype)[:, :cols]
    dy = torch.empty(rows, cols + pad, device=DEV, dtype=dtype)[:, :cols]
    dy.copy_(values[:, None].expand(-1, cols))
    mean = torch.full((rows,), 2.0, device=DEV)
    rstd = torch.full((rows,), 1e6, device=DEV)
    dx = backward(dy, x, None, mean, rstd).double()
    k = 80 + cols / 256
    exact = 0
    for row, t in zip(dx, values.tolist()):
        significand = int(math.frexp(abs(t))[0] * 2 ** 11)
        while significand % 2 == 0:
            significand //= 2
        if significand * cols < 2 ** 24:
            assert (row == 0).all(), t
            exact += 1
        else:
            assert (row.abs() <= 1e6 * (k + 2) * U * abs(t)).all(), t
    assert exact >= 3                    # the test is not empty


@pytest.mark.parametrize("cols", COLS)
def test_a_gradient_of_a_few_ulps_around_its_mean(cols):
    g = torch.Generator(device=DEV).manual_seed(cols)
    rows = 6
    dy = 1.7 + torch.randn(rows, cols, generator=g, device=DEV) * 2.0 ** -20
    x = torch.full((rows, cols), 2.0, device=DEV)
    mean, rstd = torch.full((rows,), 2.0, device=DEV), torch.full((rows,), 1e3, device=DEV)
    dx = backward(dy, x, None, mean, rstd).double()
    t = dy.double()
    want = 1e3 * (t - t.mean(1, keepdim=True))
    k = 80 + cols / 256
    assert ((dx - want).abs() <= 1e3 * (k + 2) * U * 1.71 + 4 * U * (want.abs() + 1.71e3)).all()
