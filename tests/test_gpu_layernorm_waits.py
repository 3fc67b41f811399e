"""The layer norm backward pass's bounded waits, made to run out without a
fault: cc_inject_layernorm_stall leaves out one row's copies and bounds the
launch's waits by a few milliseconds.  The CTA that waits for them gives up and
reports it; nothing is written from rows that never came: dx of the rows that
were not reached, dweight and dbias keep their contents, every other row is
exact.  The next call runs normally."""
import time

import pytest
import torch

from gradient_reduce_optimizer_gb300 import build as gbuild
from gradient_reduce_optimizer_gb300 import capi

pytestmark = pytest.mark.gpu

DEV = "cuda"
SMS = 152


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()
    capi.lib()


def call(x, dy, w, mean, rstd, dsum, dx, dw, db):
    rows, cols = x.shape
    nb = capi.cc_layernorm_backward_workspace(rows, cols)
    ws = torch.full((nb,), 0xFF, device=DEV, dtype=torch.uint8)
    capi.cc_layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, rows, cols, ws, nb, dsum=dsum)
    torch.cuda.synchronize()


# one warp a row, several, rows read twice, odd lengths, one CTA for all rows,
# one stage of rows that hardly fits
CASES = [(2000, 64, torch.bfloat16), (2000, 1024, torch.bfloat16), (700, 3072, torch.float32),
         (400, 16384, torch.bfloat16), (400, 13000, torch.float32), (3000, 1023, torch.bfloat16),
         (500, 4097, torch.float32), (7, 105, torch.float32), (12, 1024, torch.bfloat16),
         (1, 256, torch.float16)]


@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("rows,cols,dtype", CASES, ids=str)
def test_rows_that_never_come(rows, cols, dtype, at):
    row = {"first": 0, "middle": rows // 2, "last": rows - 1}[at]
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    x, dy, ds = (torch.randn(rows, cols, generator=g, device=DEV).to(dtype) for _ in range(3))
    w = torch.randn(cols, generator=g, device=DEV)
    mean = x.float().mean(1)
    rstd = (x.float().var(1, correction=0) + 1e-5).rsqrt()
    inputs = (x, dy, w, mean, rstd, ds)

    def fresh():
        return (torch.full_like(x, -7.0), torch.full_like(w, -7.0), torch.full_like(w, -7.0))

    assert capi.cc_device_status() == 0
    want = fresh()
    call(*inputs, *want)
    got = fresh()
    capi.cc_inject_layernorm_stall(row, 20000)
    t0 = time.perf_counter()
    call(*inputs, *got)
    assert time.perf_counter() - t0 < 5.0
    assert capi.cc_device_status(clear=True) == 4096
    same = (got[0] == want[0]).all(1)
    left = (got[0] == -7.0).all(1)
    assert (same | left).all() and left[row] and not same[row]
    # no more than one CTA's rows
    assert left.sum().item() <= (rows + SMS - 1) // SMS + 32
    assert (got[1] == -7.0).all() and (got[2] == -7.0).all()
    again = fresh()
    call(*inputs, *again)
    for a, b in zip(again, want):
        assert torch.equal(a, b)
    assert capi.cc_device_status() == 0


def test_arguments():
    for bad in ((-2, 100), (0, 0), (0, 2000000), (1 << 31, 100)):
        with pytest.raises(capi.CCError):
            capi.cc_inject_layernorm_stall(*bad)
    capi.cc_inject_layernorm_stall(-1, 0)
