"""What the Muon binding refuses about its tensors, before the library (which
sees addresses alone) is called: types other than the call's, slabs and
workspaces that are too small or have strides, fewer slabs than replicas."""
import pytest
import torch

from gradient_reduce_optimizer_gb300 import build as gbuild
from gradient_reduce_optimizer_gb300 import capi

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
COUNT, M, N = 2, 72, 40


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()


def refused(call, words, **kw):
    with pytest.raises(capi.CCError) as e:
        call(**kw)
    assert e.value.status == capi.CC_ERR_INVALID
    assert words in e.value.reason, e.value.reason


def ortho(**kw):
    nb = capi.cc_muon_workspace(COUNT, M, N)
    t = dict(g=torch.zeros(COUNT, M, N), out=torch.zeros(COUNT, M, N, dtype=BF16),
             workspace=torch.zeros(nb, dtype=torch.uint8), g_dtype=None)
    t.update(kw)
    capi.cc_muon_orthogonalise(t["g"], t["out"], COUNT, M, N, t["workspace"], nb,
                               g_dtype=t["g_dtype"], stream=0)


def test_orthogonalise():
    for dtype in (F32, F16):
        refused(ortho, "out is", out=torch.zeros(COUNT, M, N, dtype=dtype))
    refused(ortho, "g is", g_dtype=capi.CC_DTYPE_BF16)
    refused(ortho, "workspace", workspace=torch.zeros(999, dtype=torch.uint8))


def step(**kw):
    n, R, span = 2 * 2880 + 8, 3, 2880
    nb = capi.cc_muon_workspace(COUNT, M, N)
    t = dict(grads=[torch.zeros(n, dtype=BF16) for _ in range(R)],
             acc=[torch.zeros(n) for _ in range(R)], master=torch.zeros(n),
             momentum=torch.zeros(n), params_out=[torch.zeros(n, dtype=BF16) for _ in range(R)],
             workspace=torch.zeros(nb, dtype=torch.uint8))
    t.update({k: v(t[k]) for k, v in kw.items()})
    capi.cc_fused_dp_muon(t["grads"], t["acc"], t["master"], t["momentum"], t["params_out"], n, R,
                          [0, span], M, N, t["workspace"], nb, lr=0.1, stream=0)


def last(change):
    return lambda ts: ts[:-1] + [change(ts[-1])]


def test_step():
    for name in ("grads", "acc", "params_out"):
        refused(step, f"{name}[2] is", **{name: last(lambda t: t.to(F16))})
        refused(step, f"{name}[2] must", **{name: last(lambda t: t[1:])})
        refused(step, f"{name}[2] must",
                **{name: last(lambda t: torch.zeros(2 * t.numel(), dtype=t.dtype)[::2])})
        refused(step, "2 slabs for R=3", **{name: lambda ts: ts[:2]})
    for name in ("master", "momentum"):
        refused(step, f"{name} is", **{name: lambda t: t.to(BF16)})
        refused(step, f"{name} must", **{name: lambda t: t[1:]})
    refused(step, "workspace", workspace=lambda t: t[1:])


def test_workspace_that_does_not_fit_in_64_bits():
    """2^31 - 1 of the largest matrices are refused; the most that a call takes
    are not."""
    side = 1 << 20
    assert capi.cc_muon_workspace(65535, side, side) > 65535 * 11 * side * side
    for count, rows, cols in (((1 << 31) - 1, side, side), (1 << 22, side, side),
                              ((1 << 31) - 1, side, side // 2)):
        with pytest.raises(capi.CCError) as e:
            capi.cc_muon_workspace(count, rows, cols)
        assert e.value.status == capi.CC_ERR_INVALID and "too large" in e.value.reason
