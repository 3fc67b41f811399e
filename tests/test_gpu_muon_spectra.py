"""How accurate the orthogonalisation is, by the singular values of the matrix.

The bound is the first-order effect of the iteration's roundings, from the
singular values s_i alone.  In the singular vectors' basis the step
f(x) = a x + b x^3 + c x^5 carries a small error of X's elements (i, j) and
(j, i) on by the divided differences
    (f(s_i) - f(s_j)) / (s_i - s_j)  on their symmetric part,
    (f(s_i) + f(s_j)) / (s_i + s_j)  on the antisymmetric one,
and of the elements beyond the square by f(s_i) / s_i.  Where one of the two is
large that is about one; two small ones grow by up to a = 3.44 a step, and a
rounding of X relative to its large elements with them.  So a matrix whose norm
lies in few directions comes out less accurate than a Gaussian one.

A rounding to p bits has a root mean square of 2^-p 0.43 of the matrix (uniform
within half a unit, over significands spread logarithmically), lies evenly over
the basis and is independent of the others, so their squares add.  What is
rounded, in 11 bits unless said otherwise:
  X    in the products; in the term a X too in the last two steps' input (before
       them a low part leaves 0.06 of it: two more bits of five).  The first X is
       the matrix itself: exact in 16 bits, 8 bits and a low part of 8 in fp32;
  A    which reaches P by b + c (l_i + l_j), l being A's eigenvalues;
  P    in 8 bits in the first step of bf16 and fp32 matrices.
P reaches X by P X.  Tolerance: 1.2 times this root mean square (large sums, of
10^4 terms and more, scatter by percents), and where bf16 comes out its own
rounding, 1.7e-3, added in squares."""
import math

import pytest
import torch

from gradient_reduce_optimizer_gb300 import build as gbuild
from gradient_reduce_optimizer_gb300 import capi

pytestmark = pytest.mark.gpu

DEV = "cuda"
a, b, c = capi.MUON_COEFFS
STEPS = 5
R11 = 2.0 ** -11 * 0.43
BF16_MEAN = 1.7e-3


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()
    yield
    assert capi.cc_device_status(clear=True) == 0


def expected_error(g, first_bits):
    """The root mean square of the result's error over the result's norm.
    first_bits: 16 for bf16 and 11 for fp16 matrices, which the products read as
    they are (P in the first step is 8 and 11 bits), 8 for fp32 ones."""
    m, n = min(g.shape), max(g.shape)
    s = torch.linalg.svdvals(g.double())
    x = [s / s.norm()]
    for _ in range(STEPS):
        x.append(x[-1] * (a + b * x[-1] ** 2 + c * x[-1] ** 4))

    def derivative(v):
        i, j = v[:, None], v[None, :]
        even, odd = i * i + j * j, i * j
        return (a + b * (even + odd) + c * (even * even - odd * odd + odd * even),
                a + b * (even - odd) + c * (even * even - odd * odd - odd * even),
                a + b * v ** 2 + c * v ** 4)

    step = [derivative(v) for v in x[:STEPS]]
    ones = torch.ones(m, m, dtype=torch.float64, device=g.device)
    onward = [(ones, ones, torch.ones_like(s))]           # from after step k to the end
    for k in range(STEPS - 1, 0, -1):
        onward.insert(0, tuple(p * q for p, q in zip(step[k], onward[0])))
    square = 0.0
    for k in range(STEPS):
        v, after = x[k], onward[k]
        # the kernels expand the polynomial around A = t I in the last steps
        t = 0.25 * max(0, min(3 - (STEPS - 1 - k), k - 1))
        ca, cb = a + t * (b + t * c), b + 2 * t * c
        if k > 0:
            high, low = R11, R11 * (0.06 if k <= STEPS - 3 else 1.0)
        else:
            high = 2.0 ** -8 * 0.43 if first_bits == 8 else 0.0
            low = high * 2.0 ** -8 * 0.43
        each = v.norm() / math.sqrt(m * n)
        apart = k == 0 or k <= STEPS - 3                  # a X takes X's low part
        through_p = [(d - ca) * q if apart else d * q for d, q in zip(step[k], after)]
        through_a = [ca * q if apart else 0 * q for q in after]
        for size, way in ((high, through_p), (low, through_a)):
            square += (size * each) ** 2 * ((way[0] ** 2 + way[1] ** 2).sum() / 2 +
                                            (n - m) * (way[2] ** 2).sum())
        eig = v * v - t
        p = cb * eig + c * eig * eig
        i, j = v[:, None], v[None, :]
        p_bits = R11 if k > 0 or first_bits == 11 else 2.0 ** -8 * 0.43
        for size, way in ((R11 * eig.norm() / m, cb + c * (eig[:, None] + eig[None, :])),
                          (p_bits * p.norm() / m, 1.0)):
            square += ((size * way * (i + j) / 2 * after[0]) ** 2 +
                       (size * way * (i - j) / 2 * after[1]) ** 2).sum()
    return math.sqrt(square) / x[STEPS].norm().item()


def exact(g):
    x = g.double()
    x = x / x.norm()
    for _ in range(STEPS):
        gram = x @ x.T if x.shape[0] <= x.shape[1] else x.T @ x
        p = b * gram + c * gram @ gram
        x = a * x + (p @ x if x.shape[0] <= x.shape[1] else x @ p)
    return x


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def matrix(kind, m, n, g):
    if kind == "gauss":
        return randn(g, m, n)
    if kind.startswith("1/k^"):
        r = min(m, n)
        u, v = (torch.linalg.qr(randn(g, k, r))[0] for k in (m, n))
        return (u / torch.arange(1, r + 1, device=DEV) ** float(kind[4:])) @ v.T
    if kind == "tokens":                             # 64 tokens with a direction in common
        return (randn(g, 64, m) + randn(g, 1, m)).T @ (randn(g, 64, n) + 3 * randn(g, 1, n))
    rank, noise = kind.split(" + ")
    rank = int(rank.split()[1])
    return randn(g, m, rank) @ randn(g, rank, n) + float(noise) * randn(g, m, n)


KINDS = ["gauss", "1/k^1", "1/k^2", "1/k^3", "rank 8 + 0.05", "rank 8 + 0.003", "rank 1 + 0.05",
         "rank 1 + 0.003", "rank 1 + 0.001", "rank 1 + 0.0001", "rank 1 + 0", "tokens"]
SHAPES = [(512, 512), (200, 904), (904, 200), (96, 96), (129, 2001)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n", SHAPES)
def test_orthogonalise(m, n, kind):
    g = torch.Generator(device=DEV).manual_seed(m + n)
    for dtype, bits in ((torch.bfloat16, 16), (torch.float16, 11), (torch.float32, 8)):
        x = matrix(kind, m, n, g).to(dtype)
        out = torch.empty(m, n, device=DEV, dtype=torch.bfloat16)
        nb = capi.cc_muon_workspace(1, m, n)
        ws = torch.empty(nb, device=DEV, dtype=torch.uint8)
        capi.cc_muon_orthogonalise(x, out, 1, m, n, ws, nb, eps=0.0)
        want = exact(x)
        error = ((out.double() - want).norm() / want.norm()).item()
        assert error <= math.hypot(BF16_MEAN, 1.2 * expected_error(x, bits)), dtype


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n", SHAPES)
def test_step(m, n, kind):
    """The same without bf16 on the way out: master weights of zero, a learning
    rate of one, and the update itself (gradients of zero, so that the momentum,
    fp32, is all of it) come out as the fp32 master weights."""
    g = torch.Generator(device=DEV).manual_seed(m + n + 1)
    momentum = matrix(kind, m, n, g).flatten().contiguous()
    beta = 0.5                                       # exact, as its products are
    update = (momentum * beta * beta).view(m, n)
    master = torch.zeros(m * n, device=DEV)
    grads = [torch.zeros(m * n, device=DEV, dtype=torch.bfloat16)]
    out = [torch.empty(m * n, device=DEV, dtype=torch.bfloat16)]
    nb = capi.cc_muon_workspace(1, m, n)
    ws = torch.empty(nb, device=DEV, dtype=torch.uint8)
    capi.cc_fused_dp_muon(grads, None, master, momentum, out, m * n, 1, [0], m, n, ws, nb, lr=1.0,
                          beta=beta, eps=0.0)
    want = exact(update)
    error = ((-master.double().view(m, n) - want).norm() / want.norm()).item()
    assert error <= 1.2 * expected_error(update, 8)


# ---- a side of at most 64: fp32 --------------------------------------------------


def expected_error_small(g):
    """There every iterate is Q(A) G, Q the steps' polynomial of the first Gram
    matrix A alone, with eigenvalues l = s^2.  A's entries are off by rms 2^-24 0.43
    a rounding over chains of some 64, evenly over the eigenvectors' basis: element
    (i, j) reaches the result as the divided difference of Q at l_i and l_j times
    s_j.  Q's own entries are off by as much of Q, which is a^5 = 485 on the small
    singular values."""
    s = torch.linalg.svdvals(g.double())
    s = s / s.norm()
    eig, m = s * s, len(s)

    def polynomial(l):
        q, x = torch.ones_like(l), l
        for _ in range(STEPS):
            f = a + b * x + c * x * x
            q, x = q * f, x * f * f
        return q

    i, j = eig[:, None], eig[None, :]
    q = polynomial(eig)
    at = eig.clone().requires_grad_(True)
    slope = torch.autograd.grad(polynomial(at).sum(), at)[0]
    divided = torch.where((i - j).abs() <= 1e-7 * (i + j), ((slope[:, None] + slope) / 2),
                          (q[:, None] - q[None, :]) / (i - j))
    unit = 2.0 ** -24 * 0.43 * 8
    through_a = unit * eig.norm() / m * (divided * s[None, :]).norm()
    through_q = unit * q.norm() / math.sqrt(m)
    return (torch.hypot(through_a, through_q) / (q * s).norm()).item()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n", [(64, 200), (200, 60), (33, 70), (16, 400)])
def test_step_of_few_rows(m, n, kind):
    """In fp32, by the step.  Four times the estimate, which takes the chains'
    lengths from their order of size alone, and 1e-5 for the roundings that it leaves
    out (of G's product with Q, a few 2^-24 of the result each)."""
    g = torch.Generator(device=DEV).manual_seed(m + n + 2)
    momentum = matrix(kind, m, n, g).flatten().contiguous()
    update = (momentum * 0.25).view(m, n)
    master = torch.zeros(m * n, device=DEV)
    grads = [torch.zeros(m * n, device=DEV, dtype=torch.bfloat16)]
    out = [torch.empty(m * n, device=DEV, dtype=torch.bfloat16)]
    nb = capi.cc_muon_workspace(1, m, n)
    ws = torch.empty(nb, device=DEV, dtype=torch.uint8)
    capi.cc_fused_dp_muon(grads, None, master, momentum, out, m * n, 1, [0], m, n, ws, nb, lr=1.0,
                          beta=0.5, eps=0.0)
    want = exact(update)
    error = ((-master.double().view(m, n) - want).norm() / want.norm()).item()
    assert error <= 4 * expected_error_small(update) + 1e-5
