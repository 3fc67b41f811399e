"""What the layer norm binding refuses about its tensors: types that do not
belong together, vectors with strides, tensors that are too small.  The library
sees addresses alone, so each of these would read or write other elements than
the tensors'.  (All of it is refused before the library is called, so no GPU is
needed.)"""
import pytest
import torch

from gradient_reduce_optimizer_gb300 import build as gbuild
from gradient_reduce_optimizer_gb300 import capi

ROWS, COLS = 6, 40
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()


def rows(dtype=BF16, n=ROWS, cols=COLS):
    return torch.zeros(n, cols, dtype=dtype)


def forward(stream=None, **kw):
    t = dict(x=rows(), weight=torch.zeros(COLS), bias=torch.zeros(COLS), y=rows(),
             mean=torch.zeros(ROWS), rstd=torch.zeros(ROWS), residual=rows(), sum_out=rows())
    t.update(kw)
    capi.cc_layernorm_forward(t["x"], t["weight"], t["bias"], t["y"], t["mean"], t["rstd"], ROWS,
                              COLS, 1e-5, residual=t["residual"], sum_out=t["sum_out"],
                              stream=stream)


def backward(stream=None, **kw):
    nb = capi.cc_layernorm_backward_workspace(ROWS, COLS)
    t = dict(dy=rows(), x=rows(), weight=torch.zeros(COLS), mean=torch.zeros(ROWS),
             rstd=torch.zeros(ROWS), dx=rows(), dweight=torch.zeros(COLS), dbias=torch.zeros(COLS),
             workspace=torch.zeros(nb, dtype=torch.uint8), dsum=rows())
    t.update(kw)
    capi.cc_layernorm_backward(t["dy"], t["x"], t["weight"], t["mean"], t["rstd"], t["dx"],
                               t["dweight"], t["dbias"], ROWS, COLS, t["workspace"], nb,
                               dsum=t["dsum"], stream=stream)


def strided(t):
    """The same shape, every second element of a longer tensor."""
    return torch.zeros(2 * t.numel(), dtype=t.dtype)[::2]


def refused(call, words, **kw):
    for stream in (None, 0):         # the arguments taken in C, and in Python
        with pytest.raises(capi.CCError) as e:
            call(stream=stream, **kw)
        assert e.value.status == capi.CC_ERR_INVALID
        assert words in e.value.reason and list(kw)[0] in e.value.reason, e.value.reason


@pytest.mark.parametrize("name", ["residual", "y", "sum_out", "mean", "rstd", "bias"])
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
def test_forward_types(name, dtype):
    own = {"mean": F32, "rstd": F32, "bias": F32}.get(name, BF16)
    shape = {"mean": (ROWS,), "rstd": (ROWS,), "bias": (COLS,)}.get(name, (ROWS, COLS))
    if dtype != own:
        refused(forward, "takes it as", **{name: torch.zeros(*shape, dtype=dtype)})


@pytest.mark.parametrize("name", ["dy", "dx", "dsum", "mean", "rstd", "dweight", "dbias"])
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
def test_backward_types(name, dtype):
    own = F32 if name in ("mean", "rstd", "dweight", "dbias") else BF16
    shape = {"mean": (ROWS,), "rstd": (ROWS,), "dweight": (COLS,), "dbias": (COLS,)}.get(
        name, (ROWS, COLS))
    if dtype != own:
        refused(backward, "takes it as", **{name: torch.zeros(*shape, dtype=dtype)})


def test_vectors_with_strides():
    for name in ("weight", "bias"):
        refused(forward, "contiguous", **{name: strided(torch.zeros(COLS))})
    for name in ("weight", "dweight", "dbias"):
        refused(backward, "contiguous", **{name: strided(torch.zeros(COLS))})
    for call in (forward, backward):
        for name in ("mean", "rstd"):
            refused(call, "contiguous", **{name: strided(torch.zeros(ROWS))})


def test_tensors_that_are_too_small():
    for name in ("x", "y", "residual", "sum_out"):
        refused(forward, "holds no", **{name: rows(n=ROWS - 1)})
        refused(forward, "holds no", **{name: torch.zeros(ROWS, COLS + 5, dtype=BF16)[:, :COLS - 1]})
    for name in ("dy", "x", "dx", "dsum"):
        refused(backward, "holds no", **{name: rows(n=ROWS - 1)})
    for name in ("weight", "bias"):
        refused(forward, "contiguous", **{name: torch.zeros(COLS - 1)})
    for name in ("weight", "dweight", "dbias"):
        refused(backward, "contiguous", **{name: torch.zeros(COLS - 1)})
    for call in (forward, backward):
        for name in ("mean", "rstd"):
            refused(call, "contiguous", **{name: torch.zeros(ROWS - 1)})
    refused(backward, "contiguous", workspace=torch.zeros(100, dtype=torch.uint8))


def test_types_given_with_tensors_must_be_theirs():
    x = rows(F16)
    with pytest.raises(capi.CCError) as e:
        capi.cc_layernorm_forward(x, None, None, rows(F16), None, None, ROWS, COLS, 1e-5,
                                  act_dtype=capi.CC_DTYPE_BF16, param_dtype=capi.CC_DTYPE_F32,
                                  stream=0)
    assert "takes it as" in e.value.reason
    # bits of bf16 in a type of that width pass, as raw pointers do
    bits = rows(torch.int16)
    assert capi._rows(bits, capi.CC_DTYPE_BF16, ROWS, COLS, "x", "f") == (bits.data_ptr(), COLS)
    with pytest.raises(capi.CCError):
        capi._rows(rows(torch.int32), capi.CC_DTYPE_BF16, ROWS, COLS, "x", "f")


def test_larger_tensors_pass():
    """More rows than the call takes, and views of wider rows."""
    x = torch.zeros(ROWS + 3, COLS + 4, dtype=BF16)[:, :COLS]
    assert capi._rows(x, capi.CC_DTYPE_BF16, ROWS, COLS, "x", "f") == (x.data_ptr(), COLS + 4)
    w = torch.zeros(COLS + 9)
    assert capi._vector(w, capi.CC_DTYPE_F32, COLS, "w", "f") == w.data_ptr()
