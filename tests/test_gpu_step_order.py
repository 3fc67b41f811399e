"""A step's buckets behind kernels that let their dependents start early.

Only the first bucket of a step waits for what ran before the call; the others
are held back by it alone.  The layer norm kernels let the next launch start as
soon as they run, and their dweight and dbias may lie in any bucket's range of
a gradient slab: the step has to see them all the same.  (Buckets of 64 KiB are
a few CTAs each, resident beside the layer norm's.)"""
import pytest
import torch

from gradient_reduce_optimizer_gb300 import build as gbuild
from gradient_reduce_optimizer_gb300 import capi
from gpu_common import DEV, compare_all, host_copy, new_slabs, oracle_step, random_inputs

pytestmark = pytest.mark.gpu

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, grad_scale=1.0)
BUCKET = 1 << 16                     # bytes: 32768 elements
PER = BUCKET // 2


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()
    capi.lib()


@pytest.mark.parametrize("rows,cols", [(16384, 1024), (6000, 1000), (3000, 4096)])
def test_step_after_the_layer_norm_that_fills_its_gradients(rows, cols):
    """dweight at the start of bucket 1 and dbias in bucket 3, the layer norm's
    weight in bucket 2 of the parameters that the step writes."""
    R, n = 2, 5 * PER + 13
    gen = torch.Generator(device=DEV).manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=gen, device=DEV).to(torch.bfloat16)
    dy = torch.randn(rows, cols, generator=gen, device=DEV).to(torch.bfloat16)
    mean = x.float().mean(1)
    rstd = (x.float().var(1, correction=0) + 1e-5).rsqrt()
    dx = torch.empty_like(x)
    nb = capi.cc_layernorm_backward_workspace(rows, cols)
    ws = torch.empty(nb, device=DEV, dtype=torch.uint8)
    base = random_inputs(R, n, seed=3, step=2)
    weight = torch.randn(cols, generator=gen, device=DEV).to(torch.bfloat16)

    def run(synchronise):
        s = new_slabs([g.clone() for g in base[0]], *(t.clone() for t in base[1:]))
        for out in s.outs:
            out[2 * PER:2 * PER + cols] = weight
        w = s.outs[0][2 * PER:2 * PER + cols]
        dw, db = s.grads[1][PER:PER + cols], s.grads[0][3 * PER:3 * PER + cols]
        torch.cuda.synchronize()
        capi.cc_layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, rows, cols, ws, nb)
        if synchronise:
            torch.cuda.synchronize()
        capi.cc_fused_dp_step(s.grads, s.master, s.m, s.v, s.outs, n, R, BUCKET, step=2, **HP)
        torch.cuda.synchronize()
        return [s.master, s.m, s.v, dx.clone()] + s.grads + s.outs

    want = run(True)
    for k in range(40):
        for i, (got, ref) in enumerate(zip(run(False), want)):
            assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8)), (k, i)
    assert capi.cc_device_status() == 0


def test_two_bucket_steps_back_to_back():
    """The second bucket of a step reads what the second one of the step
    before wrote."""
    R, n, steps = 2, 2 * PER, 24
    s = new_slabs(*random_inputs(R, n, seed=5, step=2))
    grads, state, _ = host_copy(s)
    torch.cuda.synchronize()
    for k in range(steps):
        capi.cc_fused_dp_step(s.grads, s.master, s.m, s.v, s.outs, n, R, BUCKET, step=2 + k, **HP)
    torch.cuda.synchronize()
    for k in range(steps):
        outs = oracle_step(grads, state, dict(HP, step=2 + k))
    compare_all(s, state, outs)
