"""The CPython module in front of the operators on 8-bit codes: it is in use, and
where it cannot be loaded or built that is said, and the calls work without it."""
import subprocess
import sys
import warnings

import pytest
import torch

from quantized_convolution_amd import build, ops
from quantized_convolution_amd import token_ops as T

MODULE = "quantized_convolution_amd._wq8_buffers"


def plans():
    return T.QuantPlan(6, 8), T.RmsPlan(6, 8), T.Q8LinearPlan(6, 8, 16)


def forms(n, m, p):
    return n._pack_form, n._unpack_form, m._forward_form, m._backward_form, p._forward_form, p._backward_form


def test_plans_have_forms():
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert all(f is not None for f in forms(*plans()))


@pytest.fixture
def missing(monkeypatch):
    monkeypatch.setitem(sys.modules, MODULE, None)  # what makes an import of it fail
    monkeypatch.setattr(T, "_addresses", None)
    monkeypatch.setattr(T, "_form", None)


def test_a_missing_module_is_named_once(missing):
    with pytest.warns(RuntimeWarning, match="_wq8_buffers cannot be loaded"):
        n = T.QuantPlan(6, 8)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert all(f is None for f in forms(n, *plans()[1:]))
    with pytest.raises(ValueError, match="must be on a GPU"):
        T.wq8_quant_pack(n, torch.zeros(6, 8), *n.empty_codes("cpu"))


@pytest.mark.parametrize("why", ["fails", "is missing"])
def test_the_library_is_built_without_it(monkeypatch, tmp_path, why):
    lib, module = tmp_path / "lib.so", tmp_path / "module.so"
    module.write_text("of another source")
    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "BUFFERS_LIB", str(module))

    def run(cmd, **kw):
        if cmd[0] == "g++":
            if why == "is missing":
                raise FileNotFoundError("no g++")
            return subprocess.CompletedProcess(cmd, 1, "", "no header")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(subprocess, "run", run)
    with pytest.warns(RuntimeWarning, match="no g\\+\\+" if why == "is missing" else "no header"):
        assert build.build() == str(lib)
    assert lib.exists() and not module.exists()


def given_calls():
    z = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    n, m, p = plans()
    x, out, gamma, y, s, c = z(6, 8), z(6, 8), z(8), z(6, 16), z(6), z(6, 128, t=torch.int8)
    wq, sw, dw, ws, pw = z(16, 128, t=torch.int8), z(16), z(16, 8), m.empty_backward_workspace(), p.empty_backward_workspace()
    return [lambda: T.wq8_quant_pack(n, x, c, s), lambda: T.wq8_quant_unpack(n, c, s, out), lambda: T.wq8_rms_forward(m, x, gamma, y=out),
            lambda: T.wq8_rms_forward(m, x, gamma, codes=c, scales=s, want_y=False),
            lambda: T.wq8_rms_backward(m, x, x, s, gamma, dx=out, dgamma=gamma.clone(), workspace=ws),
            lambda: T.wq8_q8linear_forward(p, c, s, wq, sw, y=y),
            lambda: T.wq8_q8linear_backward(p, y, c, s, wq, sw, dx=out, dw=dw, workspace=pw)]


@pytest.mark.gpu
def test_given_buffers_take_the_short_way(monkeypatch):
    """And none of the checks in Python; without the module these answer the same calls."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    calls, made = given_calls(), []
    real = ops._Args

    def args(*a):
        made.append(1)
        return real(*a)

    monkeypatch.setattr(T, "_Args", args)
    for call in calls:
        call()
    assert not made
    monkeypatch.setitem(sys.modules, MODULE, None)
    monkeypatch.setattr(T, "_addresses", None)
    monkeypatch.setattr(T, "_form", None)
    with pytest.warns(RuntimeWarning):
        calls = given_calls()
    for call in calls:
        call()
    assert len(made) == len(calls)
