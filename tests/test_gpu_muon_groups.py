"""The orthogonalisation's list of tiles where it goes on from one group of
matrices to the next, with groups of unequal size, and the step where a matrix's
tiles are cut along K.  (A group holds 240 / t matrices of t tiles of A each: 240
of 65 a side, 24 of 1000, 6 of 2048.)  Every matrix is compared with its
definition in 64 bits, with the bounds of test_gpu_muon.py."""
import math

import pytest
import torch

from gradient_reduce_optimizer_gb300 import build as gbuild
from gradient_reduce_optimizer_gb300 import capi
from test_gpu_muon import check, check_step, exact, gen, ortho, step_inputs

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def library():
    gbuild.build()
    yield
    assert capi.cc_device_status(clear=True) == 0


# two groups, 301 and 300 matrices, wide and tall; 82 and 81, 81 and 80; 7 and 6;
# 6 and 5
@pytest.mark.parametrize("count,rows,cols", [(601, 65, 72), (601, 72, 65), (163, 500, 777),
                                             (161, 777, 300), (13, 2048, 2048), (11, 2304, 2400)])
def test_orthogonalise_groups(count, rows, cols):
    g = torch.randn(count, rows, cols, generator=gen(count), device=DEV).to(torch.bfloat16)
    first = ortho(g)
    check("out", first, exact(g))
    for _ in range(2):
        assert torch.equal(ortho(g), first)


# 25 and 24; 41 and 40; three groups, 43, 42 and 42
@pytest.mark.parametrize("count,rows,cols", [(49, 1000, 1001), (81, 521, 1023), (127, 530, 600)])
def test_step_groups(count, rows, cols):
    s = step_inputs(2, count, rows, cols, count, gap=8)
    check_step(s, rows, cols, lr=1e-3, beta=0.95, nesterov=True, weight_decay=0.01,
               update_scale=0.2 * math.sqrt(max(rows, cols)), grad_scale=2.0)


@pytest.mark.parametrize("count,rows,cols", [(1, 2900, 2830), (1, 2824, 4099), (2, 200, 3328),
                                             (1, 3001, 151), (3, 1500, 90)])
def test_step_with_tiles_cut_along_k(count, rows, cols):
    s = step_inputs(2, count, rows, cols, rows, gap=8)
    check_step(s, rows, cols, lr=1e-3, beta=0.95, nesterov=True, weight_decay=0.01,
               update_scale=0.2 * math.sqrt(max(rows, cols)), grad_scale=2.0)
