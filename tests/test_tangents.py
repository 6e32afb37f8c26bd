"""Forward-mode tangents are refused by every operator's function, on the long way
through the checks and on the short one: none would come out."""
import pytest
import torch
import torch.autograd.forward_ad as fw

from quantized_convolution_amd import ops as O
from quantized_convolution_amd import token_ops as T

I8 = torch.int8


def dual(t):
    return fw.make_dual(t.clone(), torch.ones_like(t))


def calls(dev):
    """(call, buffer that carries a tangent): the call with that buffer as f gives it, every buffer being given."""
    z = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device=dev)  # noqa: E731
    n, m, p = T.QuantPlan(6, 8), T.RmsPlan(6, 8), T.Q8LinearPlan(6, 8, 16)
    g, lin = O.NormPlan(2, 8, 3, 5, groups=2), O.LinearPlan(6, 8, 16)
    x, out, gamma, y, s, c = z(6, 8), z(6, 8), z(8), z(6, 16), z(6), z(6, 128, t=I8)
    wq, sw, sx, dw, w, o = z(16, 128, t=I8), z(16), z(6), z(16, 8), z(16, 8), z(6, 16)
    img, st, dx2 = z(2, 3, 5, 8), z(2, 2), z(2, 3, 5, 8)
    wsb = lambda p: p.empty_backward_workspace(dev)  # noqa: E731
    return [
        (lambda f: T.wq8_quant_pack(n, f(x), c, s), "x"), (lambda f: T.wq8_quant_unpack(n, c, f(s), x), "scales"),
        (lambda f: T.wq8_rms_forward(m, f(x), gamma, y=out), "x"), (lambda f: T.wq8_rms_forward(m, x, f(gamma), y=out), "gamma"),
        (lambda f: T.wq8_rms_backward(m, f(x), x, s, dx=out, workspace=wsb(m)), "dy"),
        (lambda f: T.wq8_q8linear_forward(p, c, f(sx), wq, sw, y=y), "sx"),
        (lambda f: T.wq8_q8linear_forward(p, c, sx, wq, sw, None, f(o), y=y), "residual"),
        (lambda f: T.wq8_q8linear_backward(p, f(y), c, sx, wq, sw, dx=out, dw=dw, workspace=wsb(p)), "dy"),
        (lambda f: O.wq8_norm_forward(g, f(img), y=dx2), "x"), (lambda f: O.wq8_norm_backward(g, img, img, f(st), st, dx=dx2), "mean"),
        (lambda f: O.wq8_linear_forward(lin, x, f(w), y=y), "w"), (lambda f: O.wq8_linear_backward(lin, f(y), x, w, dx=out, dw=dw), "dy"),
    ]


def refused(dev, without):
    for call, name in calls(dev):
        with fw.dual_level():
            with pytest.raises(ValueError, match=f"^{name} carries a tangent"):
                call(dual)
            with torch.no_grad(), pytest.raises(ValueError, match=f"^{name} carries a tangent"):
                call(dual)
            without(lambda: call(lambda t: t))  # a level alone is no reason
            without(lambda: call(lambda t: fw.unpack_dual(dual(t)).primal))


def test_tangents_are_refused():
    def without(call):
        with pytest.raises(ValueError, match="must be on a GPU"):
            call()

    refused("cpu", without)


@pytest.mark.gpu
def test_tangents_are_refused_on_the_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    refused("cuda", lambda call: call())
