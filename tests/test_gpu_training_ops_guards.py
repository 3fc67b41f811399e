"""The layer norm and Muon calls write nothing outside their tensors, let nothing
from outside into their results, and allocate nothing.  Every tensor, workspace
included, ends exactly where the call says, between two bands of bytes 0xFF
(NaN in every type)."""
import pytest
import torch

from gradient_reduce_optimizer_gb300 import build as gbuild
from gradient_reduce_optimizer_gb300 import capi

pytestmark = pytest.mark.gpu

DEV = "cuda"
GUARD = 512                   # keeps a workspace 256-byte aligned


@pytest.fixture(scope="module", autouse=True)
def library():
    gbuild.build()
    yield
    assert capi.cc_device_status(clear=True) == 0


class Guarded:
    def __init__(self):
        self.all = []

    def __call__(self, name, shape, dtype, fill=None, shift=0):
        """A tensor between bands, `shift` elements off a 256-byte boundary."""
        size = torch.empty(0, dtype=dtype).element_size()
        n = 1
        for d in shape:
            n *= d
        at = GUARD + shift * size
        buf = torch.full((at + n * size + GUARD,), 0xFF, dtype=torch.uint8, device=DEV)
        t = buf[at:at + n * size].view(dtype).view(*shape)
        if fill is not None:
            t.copy_(fill)
        self.all.append((name, buf, at, n * size))
        return t

    def check(self):
        torch.cuda.synchronize()
        for name, buf, at, size in self.all:
            assert (buf[:at] == 0xFF).all(), f"{name}: bytes before it changed"
            assert (buf[at + size:] == 0xFF).all(), f"{name}: bytes after it changed"


LN = [(1, 1), (3, 7), (5, 40), (17, 257), (33, 768), (64, 1024), (333, 1023), (7, 4099), (2, 8200),
      (5, 16384), (3, 16383), (2, 16400), (160, 20001), (2000, 64), (1000, 61), (400, 3000)]


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("rows,cols", LN)
def test_layernorm(rows, cols, dtype, shift):
    g = torch.Generator(device=DEV).manual_seed(rows + cols)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    for par in (dtype, torch.float32):
        t = Guarded()
        x, res, dy, ds = (t(n, (rows, cols), dtype, randn(rows, cols), shift)
                          for n in ("x", "residual", "dy", "dsum"))
        w, b = (t(n, (cols,), par, 1 + 0.1 * randn(cols), shift) for n in ("weight", "bias"))
        y, s, dx = (t(n, (rows, cols), dtype, shift=shift) for n in ("y", "sum_out", "dx"))
        mean, rstd = (t(n, (rows,), torch.float32) for n in ("mean", "rstd"))
        dw, db = (t(n, (cols,), par, shift=shift) for n in ("dweight", "dbias"))
        nb = capi.cc_layernorm_backward_workspace(rows, cols)
        ws = t("workspace", (nb,), torch.uint8)
        capi.cc_layernorm_forward(x, w, b, y, mean, rstd, rows, cols, 1e-5, residual=res,
                                  sum_out=s)
        capi.cc_layernorm_backward(dy, s, w, mean, rstd, dx, dw, db, rows, cols, ws, nb, dsum=ds)
        t.check()
        for r in (y, s, mean, rstd, dx, dw, db):
            assert torch.isfinite(r).all()


MUON = [(1, 1, 1), (3, 5, 7), (2, 64, 200), (2, 100, 60), (2, 65, 65), (2, 129, 257), (3, 257, 129),
        (2, 128, 128), (1, 777, 1001), (2, 1001, 333), (1, 2900, 2830), (2, 200, 3328), (250, 72, 65)]


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("count,rows,cols", MUON)
def test_orthogonalise(count, rows, cols, dtype, shift):
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    t = Guarded()
    x = t("g", (count, rows, cols), dtype,
          torch.randn(count, rows, cols, generator=g, device=DEV), shift)
    out = t("out", (count, rows, cols), torch.bfloat16, shift=shift)
    nb = capi.cc_muon_workspace(count, rows, cols)
    ws = t("workspace", (nb,), torch.uint8)
    capi.cc_muon_orthogonalise(x, out, count, rows, cols, ws, nb)
    t.check()
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("R", [1, 3, 16])
@pytest.mark.parametrize("count,rows,cols", MUON)
def test_step(count, rows, cols, R):
    """The slabs end with the last matrix's last element."""
    if count > capi.CC_MUON_MAX_MATRICES:
        count = capi.CC_MUON_MAX_MATRICES
    g = torch.Generator(device=DEV).manual_seed(rows + cols + R)
    span = (rows * cols + 7) // 8 * 8
    n = span * (count - 1) + rows * cols

    def randn():
        return torch.randn(n, generator=g, device=DEV)

    t = Guarded()
    grads = [t(f"grads[{r}]", (n,), torch.bfloat16, randn()) for r in range(R)]
    acc = [t(f"acc[{r}]", (n,), torch.float32, randn()) for r in range(R)]
    master, momentum = (t(k, (n,), torch.float32, randn()) for k in ("master", "momentum"))
    outs = [t(f"params_out[{r}]", (n,), torch.bfloat16, randn()) for r in range(R)]
    nb = capi.cc_muon_workspace(count, rows, cols)
    ws = t("workspace", (nb,), torch.uint8)
    for with_acc in (None, acc):
        capi.cc_fused_dp_muon(grads, with_acc, master, momentum, outs, n, R,
                              [span * i for i in range(count)], rows, cols, ws, nb, lr=1e-3)
    t.check()
    for r in [master, momentum] + outs:
        assert torch.isfinite(r).all()


def test_nothing_is_allocated():
    """The device's free memory stays as it is over calls of sizes not seen
    before (the kernels themselves are loaded by then)."""
    def calls(rows, cols, count, m, k):
        x = [torch.randn(rows, cols, device=DEV) for _ in range(4)]
        v = [torch.ones(cols, device=DEV) for _ in range(4)]
        s = [torch.empty(rows, device=DEV) for _ in range(2)]
        nb = capi.cc_layernorm_backward_workspace(rows, cols)
        ws = torch.empty(nb, device=DEV, dtype=torch.uint8)
        g = torch.randn(count, m, k, device=DEV)
        out = torch.empty(count, m, k, device=DEV, dtype=torch.bfloat16)
        n = count * m * k
        slabs = [torch.zeros(n, device=DEV) for _ in range(2)]
        params = [torch.zeros(n, device=DEV, dtype=torch.bfloat16)]
        nm = capi.cc_muon_workspace(count, m, k)
        wm = torch.empty(nm, device=DEV, dtype=torch.uint8)
        torch.cuda.synchronize()
        free = torch.cuda.mem_get_info()[0]
        capi.cc_layernorm_forward(x[0], v[0], v[1], x[1], *s, rows, cols, 1e-5)
        capi.cc_layernorm_backward(x[2], x[0], v[0], *s, x[3], v[2], v[3], rows, cols, ws, nb)
        capi.cc_muon_orthogonalise(g, out, count, m, k, wm, nm)
        capi.cc_fused_dp_muon([out.view(-1)], None, *slabs, params, n, 1,
                              [i * m * k for i in range(count)], m, k, wm, nm, lr=1e-3)
        torch.cuda.synchronize()
        return free - torch.cuda.mem_get_info()[0]

    calls(1000, 1024, 2, 128, 256)
    assert [calls(3000, 1024, 4, 264, 512), calls(5000, 1024, 3, 512, 776)] == [0, 0]
