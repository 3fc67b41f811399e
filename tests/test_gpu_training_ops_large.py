"""The layer norm and Muon calls on tensors whose offsets pass 2^32 elements.
Rows, matrices and offsets below, at and above 2^31 and 2^32 elements are compared
with the definitions in 64 bits; the column sums are compared whole."""
import gc

import pytest
import torch

from gradient_reduce_optimizer_gb300 import build as gbuild
from gradient_reduce_optimizer_gb300 import capi
from test_gpu_layernorm import check_forward, within
from test_gpu_muon import check, check_step, exact

pytestmark = pytest.mark.gpu

DEV = "cuda"
U32 = 2.0 ** -24


@pytest.fixture(autouse=True)
def memory():
    gbuild.build()
    if torch.cuda.mem_get_info()[1] < 120 << 30:
        pytest.skip("120 GiB of device memory")
    yield
    gc.collect()
    torch.cuda.empty_cache()
    assert capi.cc_device_status(clear=True) == 0


def filled(rows, cols, seed):
    """bf16 rows from a block of random ones, each with a factor of its own."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    block = torch.randn(4096, cols, generator=g, device=DEV).to(torch.bfloat16)
    t = torch.empty(rows, cols, device=DEV, dtype=torch.bfloat16)
    scale = (1 + torch.arange(rows, device=DEV) % 7).to(torch.bfloat16)
    for i in range(0, rows, 4096):
        n = min(4096, rows - i)
        torch.mul(block[:n], scale[i:i + n, None], out=t[i:i + n])
    return t


@pytest.mark.parametrize("cols", [16384, 16383, 1000])
def test_layernorm(cols):
    rows = (1 << 32) // cols + 5
    x = filled(rows, cols, 1)
    w = 1 + 0.1 * torch.randn(cols, device=DEV)
    b = 0.1 * torch.randn(cols, device=DEV)
    y = torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    capi.cc_layernorm_forward(x, w, b, y, mean, rstd, rows, cols, 1e-5)
    at = torch.tensor(sorted({0, 1, (1 << 31) // cols, (1 << 31) // cols + 1, rows // 2 + 1,
                              rows - 6, rows - 5, rows - 2, rows - 1}), device=DEV)
    check_forward(x[at], w, b, 1e-5, None, y[at], None, mean[at], rstd[at])
    dy, dx = y, torch.empty_like(x)                  # the result as a gradient
    dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    nb = capi.cc_layernorm_backward_workspace(rows, cols)
    ws = torch.empty(nb, device=DEV, dtype=torch.uint8)
    capi.cc_layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, rows, cols, ws, nb)
    h = (x[at].double() - mean[at].double()[:, None]) * rstd[at].double()[:, None]
    t = dy[at].double() * w.double()
    r = rstd[at].double()[:, None]
    want = r * (t - t.mean(1, keepdim=True) - h * (t * h).mean(1, keepdim=True))
    tol = r * 200 * U32 * (t.abs().amax(1, keepdim=True) * (1 + h.abs())) + 2.0 ** -8 * want.abs()
    within("dx", dx[at], want, tol)
    sums = torch.zeros(4, cols, device=DEV, dtype=torch.float64)
    for i in range(0, rows, 8192):
        n = slice(i, min(i + 8192, rows))
        d = dy[n].double()
        e = d * ((x[n].double() - mean[n].double()[:, None]) * rstd[n].double()[:, None])
        sums += torch.stack([e.sum(0), e.abs().sum(0), d.sum(0), d.abs().sum(0)])
    k = (96 + rows / 304 + 16) * U32                 # a column's chain of additions
    within("dweight", dw, sums[0], 2 * k * sums[1])
    within("dbias", db, sums[2], k * sums[3])


def test_orthogonalise():
    count, m = (1 << 32) // (1 << 20) + 3, 1024
    g = filled(count * m, m, 2).view(count, m, m)
    out = torch.empty_like(g)
    nb = capi.cc_muon_workspace(count, m, m)
    ws = torch.empty(nb, device=DEV, dtype=torch.uint8)
    capi.cc_muon_orthogonalise(g, out, count, m, m, ws, nb)
    at = [0, 2047, 2048, 2049, 4094, 4095, 4096, count - 1]
    check("out", out[at], exact(g[at]), elements=False)


@pytest.mark.parametrize("rows,cols", [(200, 264), (48, 264), (131, 201)])
def test_step_at_the_end_of_a_long_slab(rows, cols):
    span = (rows * cols + 7) // 8 * 8
    n = (1 << 32) + 4 * span + 5
    offsets = [(1 << 31) - 8, (1 << 32) - span, (1 << 32), (1 << 32) + 2 * span + 8]
    gen = torch.Generator(device=DEV).manual_seed(rows)
    ends = [(o, o + rows * cols) for o in offsets]

    def slab(sigma, dtype):
        t = torch.zeros(n, device=DEV, dtype=dtype)
        for lo, hi in ends:
            t[lo:hi] = torch.randn(hi - lo, generator=gen, device=DEV) * sigma
        return t

    grads = [slab(1e-3, torch.bfloat16)]
    master, momentum = slab(0.02, torch.float32), slab(1e-3, torch.float32)
    outs = [torch.full((n,), 3.0, device=DEV, dtype=torch.bfloat16)]
    before = [(master[lo:hi].clone(), momentum[lo:hi].clone(), grads[0][lo:hi].clone())
              for lo, hi in ends]
    nb = capi.cc_muon_workspace(len(offsets), rows, cols)
    ws = torch.empty(nb, device=DEV, dtype=torch.uint8)
    capi.cc_fused_dp_muon(grads, None, master, momentum, outs, n, 1, offsets, rows, cols, ws, nb,
                          lr=1e-2, weight_decay=0.1)
    # the same matrices in a short slab
    short = [o * span for o in range(len(offsets))]
    m = span * len(offsets)
    s = dict(grads=[torch.zeros(m, device=DEV, dtype=torch.bfloat16)], acc=None,
             master=torch.zeros(m, device=DEV), momentum=torch.zeros(m, device=DEV),
             outs=[torch.full((m,), 3.0, device=DEV, dtype=torch.bfloat16)], n=m, offsets=short)
    for o, (w, u, g) in zip(short, before):
        for to, value in ((s["master"], w), (s["momentum"], u), (s["grads"][0], g)):
            to[o:o + rows * cols] = value
    check_step(s, rows, cols, lr=1e-2, beta=0.95, nesterov=True, weight_decay=0.1, update_scale=1.0,
               grad_scale=1.0)
    for o, (lo, hi) in zip(short, ends):
        for got, want in ((master, s["master"]), (momentum, s["momentum"]), (outs[0], s["outs"][0])):
            assert torch.equal(got[lo:hi], want[o:o + rows * cols])
    # and nothing else: the elements beside them, and all of them counted
    assert int((outs[0] != 3.0).sum()) == int((s["outs"][0] != 3.0).sum())
    assert int((master != 0).sum()) == int((s["master"] != 0).sum())
