"""Layer norm of rows that are constant, or nearly so, at a small eps: rstd is
then up to 1 / sqrt(eps) = 10^6, and what the mean is off by, an ulp of it, would
show in y as a good part of the weight.

Tolerances.  With u = 2^-24 and a row's sum a chain of at most k = 80 + cols / 256
additions (a thread's elements, the trees), the first mean m is off by at most
D = (k + 2) u max|x|.  The deviations from it are exact for a row that lies within
a factor of two of its mean (Sterbenz), at most D + max|x - mean| = E in size, and
their mean c is off by at most (k + 2) u E.  Hence
  mean   (k + 2) u E, and the rounding of m + c;
  d - c  (k + 2) u E + 2 u |d| for each element's true deviation d;
  var    the two quotients and the product: 3 (k + 4) u E^2, and the same of
         the true variance;
  rstd   half of var's error relative to var + eps, and its own rounding;
  y      weight times (d - c's error times rstd, and |d| times rstd's), the
         roundings of y's own operations and of its type (in fp16's subnormals
         half of 2^-24)."""
import itertools

import pytest
import torch

from gradient_reduce_optimizer_gb300 import build as gbuild
from gradient_reduce_optimizer_gb300 import capi

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
EPS = 1e-12
HALF_TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()


def check(x, w, b):
    """x: rows x cols on the device, possibly with a row stride."""
    rows, cols = x.shape
    y = torch.empty(rows, cols, device=DEV, dtype=x.dtype)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    capi.cc_layernorm_forward(x, w, b, y, mean, rstd, rows, cols, EPS)
    k = 80 + cols / 256
    v = x.double()
    m = v.mean(1, keepdim=True)
    d = v - m
    var = d.square().mean(1, keepdim=True)
    E = (k + 2) * U * v.abs().amax(1, keepdim=True) + d.abs().amax(1, keepdim=True)
    c_err = (k + 2) * U * E
    assert ((mean.double()[:, None] - m).abs() <= c_err + U * m.abs()).all()
    r = (var + EPS).rsqrt()
    r_err = r * (0.5 * 3 * (k + 4) * U * (E.square() + var) / (var + EPS) + 4 * U)
    assert ((rstd.double()[:, None] - r).abs() <= r_err).all()
    d_err = c_err + 2 * U * d.abs()
    wd, bd = w.double(), b.double()
    want = d * r * wd + bd
    tol = (wd.abs() * (d_err * (r + r_err) + d.abs() * r_err + 4 * U * d.abs() * r)
           + 4 * U * (want.abs() + bd.abs()))
    tol = tol + HALF_ULP[x.dtype] * (want.abs() + tol) + HALF_TINY[x.dtype]
    over = ((y.double() - want).abs() - tol).max().item()
    assert over <= 0, f"y is {over:.3g} over its bound"


# rows in vectors (a warp, a CTA), element by element (a warp, a CTA), and longer
# than both; odd quotients and even ones
COLS = [41, 47, 96, 600, 1000, 1001, 1023, 3000, 5001, 8200, 16384, 16383, 16400, 20001]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("cols", COLS)
def test_constant_rows(cols, dtype):
    g = torch.Generator(device=DEV).manual_seed(cols)
    values = torch.tensor([3.0, -3.0, 0.1, 7.3, -1.7, 1e-3, 0.0, 1 / 3], device=DEV).to(dtype)
    x = values[:, None].expand(-1, cols).contiguous()
    w = 1 + 0.2 * torch.randn(cols, generator=g, device=DEV)
    b = 0.2 * torch.randn(cols, generator=g, device=DEV)
    check(x, w, b)
    off = torch.empty(len(values), cols + 3, device=DEV, dtype=dtype)[:, :cols]
    off.copy_(x)
    check(off, w, b)


@pytest.mark.parametrize("cols", COLS)
def test_rows_with_a_deviation_of_a_few_ulps(cols):
    g = torch.Generator(device=DEV).manual_seed(cols + 1)
    w = 1 + 0.2 * torch.randn(cols, generator=g, device=DEV)
    b = 0.2 * torch.randn(cols, generator=g, device=DEV)
    rows = []
    for value, ulps in itertools.product((3.0, -1.7, 0.1, 5.9), (1, 4, 30)):
        noise = torch.randn(cols, generator=g, device=DEV) * ulps * 2.0 ** -23 * abs(value)
        rows.append(value + noise)
    check(torch.stack(rows), w, b)


def test_one_element_apart():
    """All of a row but its last element the same."""
    for cols in (47, 1000, 5001, 20001):
        x = torch.full((3, cols), 2.9, device=DEV)
        x[0, -1] += 2.0 ** -20
        x[1, 0] -= 2.0 ** -21
        x[2, cols // 2] += 1e-3
        check(x, torch.ones(cols, device=DEV), torch.zeros(cols, device=DEV))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("cols", COLS)
def test_the_mean_of_a_row_whose_sum_is_exact(cols, dtype):
    """Integers: every partial sum is one below 2^24, so the mean is off by the
    quotient's roundings alone (1 / cols' and the product's), however small it is
    next to the elements, and in rows that vary little too."""
    g = torch.Generator(device=DEV).manual_seed(cols + 2)
    x = torch.randint(-100, 101, (40, cols), generator=g, device=DEV).float()
    x[20:] = 100 + torch.randint(-1, 2, (20, cols), generator=g, device=DEV)
    x = x.to(dtype)
    mean = torch.empty(40, device=DEV)
    capi.cc_layernorm_forward(x, None, None, torch.empty_like(x), mean, None, 40, cols, 1e-5)
    want = x.double().mean(1)
    error = (mean.double() - want).abs()
    assert (error[:20] <= 2.01 * U * want[:20].abs()).all()
    # corrected by the deviations' mean, itself within (80 + cols / 256) u of them
    assert (error[20:] <= U * want[20:].abs() + 2 * (80 + cols / 256) * U).all()
