"""The extension module that takes the layer norm calls' arguments is a faster
way in, not a condition: without a compiler for it the build goes through, and
without it the binding calls the library itself."""
import os
import warnings

import pytest
import torch

from gradient_reduce_optimizer_gb300 import build as gbuild
from gradient_reduce_optimizer_gb300 import capi


@pytest.fixture(autouse=True)
def built():
    gbuild.build()


def test_the_build_goes_through_without_a_compiler_for_it(tmp_path, monkeypatch, capsys):
    calls = tmp_path / "_calls.so"
    monkeypatch.setattr(gbuild, "CALLS", str(calls))
    calls.write_bytes(b"of older sources")
    os.utime(calls, (0, 0))
    for compiler in ("no-such-compiler", "false"):
        monkeypatch.setenv("CC", compiler)
        monkeypatch.setenv("CXX", compiler)
        assert gbuild.build() == gbuild.LIBRARY
        assert not calls.exists()
    assert "not built" in capsys.readouterr().err
    monkeypatch.delenv("CC")
    monkeypatch.delenv("CXX")
    gbuild.build()
    assert calls.exists()


@pytest.mark.parametrize("there", [False, True])
def test_the_binding_works_without_it(there, tmp_path, monkeypatch):
    """Where it was not built, and where what is there cannot be loaded."""
    seen = []

    class Library:
        cc_layernorm_forward = staticmethod(lambda *a: seen.append(a) or 0)
        cc_layernorm_backward = staticmethod(lambda *a: seen.append(a) or 0)

    monkeypatch.setattr(capi, "_CALLS", None)
    monkeypatch.setattr(capi, "__file__", str(tmp_path / "capi.py"))
    if there:
        (tmp_path / "_calls.so").write_bytes(b"no module")
    monkeypatch.setattr(capi, "lib", lambda: Library)
    monkeypatch.setattr(capi, "_stream", lambda s: 77)
    x, y = (torch.zeros(4, 16, dtype=torch.float16) for _ in range(2))
    w, m = torch.zeros(16), torch.zeros(4)
    with warnings.catch_warnings(record=True) as caught:
        warnings.simplefilter("always")
        capi.cc_layernorm_forward(x, w, None, y, m, None, 4, 16, 1e-5)
    assert len(caught) == there
    capi.cc_layernorm_backward(y, x, w, m, m, y, None, None, 4, 16)
    assert seen[0][0] == x.data_ptr() and seen[0][-3:] == (capi.CC_DTYPE_F16, capi.CC_DTYPE_F32, 77)
    assert seen[1][0] == y.data_ptr() and seen[1][-1] == 77
