"""The bounded waits of the orthogonalisation's products, made to run out without
a fault: cc_inject_muon_stall keeps one matrix of a batch from its second product
and bounds the launch's waits by some milliseconds.  Every cluster that comes to
that matrix, or to what such a cluster left undone, gives up and reports it; no
copy is in flight then, the launch returns, what was not computed keeps its
contents, what was is exact, and the next call runs normally."""
import time

import pytest
import torch

from gradient_reduce_optimizer_gb300 import build as gbuild
from gradient_reduce_optimizer_gb300 import capi

pytestmark = pytest.mark.gpu

DEV = "cuda"
PRODUCER, REST = 256, 512 | 1024 | 2048
# one tile, several, more tiles than clusters, tiles cut along K, tall and wide
SHAPES = [(1, 100, 100), (5, 128, 192), (40, 256, 300), (3, 777, 1001), (2, 200, 3328),
          (3, 1001, 333)]


@pytest.fixture(scope="module", autouse=True)
def library():
    gbuild.build()
    yield
    assert capi.cc_device_status(clear=True) == 0


@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("count,rows,cols", SHAPES)
def test_orthogonalise(count, rows, cols, last):
    g = torch.randn(count, rows, cols, device=DEV,
                    generator=torch.Generator(device=DEV).manual_seed(rows))
    nb = capi.cc_muon_workspace(count, rows, cols)
    ws = torch.empty(nb, device=DEV, dtype=torch.uint8)

    def call():
        out = torch.full(g.shape, 3.0, device=DEV, dtype=torch.bfloat16)
        capi.cc_muon_orthogonalise(g, out, count, rows, cols, ws, nb)
        torch.cuda.synchronize()
        return out

    assert capi.cc_device_status() == 0
    want = call()
    stalled = count - 1 if last else 0
    capi.cc_inject_muon_stall(stalled, 20000)
    t0 = time.perf_counter()
    got = call()
    assert time.perf_counter() - t0 < 5.0
    status = capi.cc_device_status(clear=True)
    assert status & PRODUCER and not status & ~(PRODUCER | REST), status
    assert (got[stalled] == 3.0).all()
    assert ((got == want) | (got == 3.0)).all()
    assert torch.equal(call(), want)
    assert capi.cc_device_status() == 0


def test_step():
    count, rows, cols, R = 3, 264, 200, 2
    span = rows * cols
    n = span * count
    gen = torch.Generator(device=DEV).manual_seed(1)
    grads = [torch.randn(n, generator=gen, device=DEV).to(torch.bfloat16) for _ in range(R)]
    master0, momentum0 = (torch.randn(n, generator=gen, device=DEV) for _ in range(2))
    nb = capi.cc_muon_workspace(count, rows, cols)
    ws = torch.empty(nb, device=DEV, dtype=torch.uint8)

    def call():
        master, momentum = master0.clone(), momentum0.clone()
        outs = [torch.full((n,), 3.0, device=DEV, dtype=torch.bfloat16) for _ in range(R)]
        capi.cc_fused_dp_muon(grads, None, master, momentum, outs, n, R,
                              [span * i for i in range(count)], rows, cols, ws, nb, lr=0.1)
        torch.cuda.synchronize()
        return master, momentum, outs

    master, momentum, outs = call()
    capi.cc_inject_muon_stall(1, 20000)
    m2, mom2, outs2 = call()
    status = capi.cc_device_status(clear=True)
    assert status & PRODUCER and not status & ~(PRODUCER | REST), status
    assert torch.equal(mom2, momentum)                # a pass of its own, before
    one = slice(span, 2 * span)
    assert torch.equal(m2[one], master0[one])
    assert ((m2 == master) | (m2 == master0)).all()
    for a, b in zip(outs2, outs):
        assert (a[one] == 3.0).all() and ((a == b) | (a == 3.0)).all()
    again = call()
    assert torch.equal(again[0], master)
    assert capi.cc_device_status() == 0


def test_arguments():
    for bad in ((-2, 100), (0, 0), (0, 2000000)):
        with pytest.raises(capi.CCError):
            capi.cc_inject_muon_stall(*bad)
    capi.cc_inject_muon_stall(-1, 0)
