"""A feed forward that is given its own buffers: what it returned from a call, or
from a backward."""
import pytest
import torch

import quantized_convolution_amd as q
from quantized_convolution_amd.token_block import Q8FeedForward

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
ROWS, C, D = 77, 200, 520


@pytest.fixture(scope="module", autouse=True)
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.load()


def make(dtype, rows=ROWS, **kw):
    g = torch.Generator().manual_seed(rows)
    r = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
    w = {"gamma": 1 + 0.1 * r(C), "w1": (r(D, C) / C ** 0.5).to(dtype), "w2": (r(C, D) / D ** 0.5).to(dtype), "b1": 0.1 * r(D),
         "b2": 0.1 * r(C)}
    return [Q8FeedForward(w, rows, C, dtype, **kw) for _ in range(2)], r(rows, C).to(dtype), r(rows, C).to(dtype)


def equal(a, b):
    return a.keys() == b.keys() and all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows", [1, ROWS])
def test_its_own_output(rows, dtype):
    """The gradients are those of the last call, whichever buffer its input came in."""
    (ff, fresh), x, dout = make(dtype, rows)
    once = ff(x).clone()
    twice = ff(ff(x))
    want = fresh(once)
    assert torch.equal(twice, want)
    assert torch.equal(ff.stream, once)
    assert equal(ff.backward(dout), fresh.backward(dout))
    # as rows of a view, and a third time
    assert torch.equal(ff(ff(ff(x)).view(rows, C)), fresh(want.clone()))
    assert equal(ff.backward(dout), fresh.backward(dout))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_its_own_output_as_residual(dtype):
    (ff, fresh), x, dout = make(dtype)
    once = ff(x).clone()
    assert torch.equal(ff(x, ff(x)), fresh(x, once))
    assert equal(ff.backward(dout), fresh.backward(dout))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_its_own_gradient(dtype):
    """As an input, and as the gradient that the next backward is given."""
    (ff, fresh), x, dout = make(dtype)
    ff(x)
    dx = ff.backward(dout)["x"]
    kept = dx.clone()
    assert torch.equal(ff(dx), fresh(kept))
    assert equal(ff.backward(dout), fresh.backward(dout))
    ff(x), fresh(x)
    dx = ff.backward(dout)["x"]
    kept = dx.clone()  # the next backward writes its own over it
    assert equal(ff.backward(dx), fresh.backward(kept))


def test_its_own_output_without_training():
    (ff, fresh), x, _ = make(BF, train=False)
    once = ff(x).clone()
    assert torch.equal(ff(ff(x)), fresh(once))


def test_its_own_output_in_a_graph():
    (ff, fresh), x, dout = make(BF)
    for _ in range(2):
        ff(ff(x)), ff.backward(dout)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ff(ff(x))
        grads = ff.backward(dout)
    for seed in range(4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(ROWS, C, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = fresh(fresh(x).clone())
        assert torch.equal(out, want) and equal(grads, fresh.backward(dout))
        torch.cuda.synchronize()


def test_parts_of_its_own_output_are_refused():
    """As parts of any tensor are: nothing is spread or turned to the block's shape."""
    (ff, _), x, _ = make(F32)
    out = ff(x)
    for part, what in ((out[:1], "x must have shape"), (out[0], "x must have shape"), (out.view(C, ROWS).T, "x must be contiguous"),
                       (out.view(torch.int32), "x must be torch.float32"), (None, "x is required")):
        with pytest.raises(ValueError, match=what):
            ff(part)


def test_what_a_block_holds():
    """33.5 bytes a value of the stream in bf16 for an inner width of 4 C, 9.5 of them codes for the backward; one number a row."""
    rows, width = 64, 256
    z = lambda *s, t=BF: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    w = {"gamma": z(width, t=F32), "w1": z(4 * width, width), "w2": z(width, 4 * width), "b1": z(4 * width, t=F32), "b2": z(width, t=F32)}
    ff = Q8FeedForward(w, rows, width)
    size = lambda *ts: sum(t.numel() * t.element_size() for t in ts)  # noqa: E731
    codes = size(ff.a[0], ff.uq[0], *ff.z)
    assert codes == 9.5 * rows * width
    assert size(ff.a[1], ff.uq[1], ff.rstd) == 3 * 4 * rows
    assert size(ff.h, ff.u, ff.out, ff.du, ff.da, ff.dx) == 24 * rows * width
    own = [t for v in vars(ff).values() for t in (v if isinstance(v, tuple) else (v,)) if isinstance(t, torch.Tensor)]
    assert size(*own) == 33.5 * rows * width + 12 * rows + size(ff.ws, *ff.w1, *ff.w2)
