"""Which calls of the operators on 8-bit codes may take the short way through the
checks: those that make nothing. What it returns is what the longer one does."""
import pytest
import torch

from quantized_convolution_amd import token_ops as T

F32, I8 = torch.float32, torch.int8


@pytest.fixture
def short(monkeypatch):
    """Counts the calls that would be made on the short way, and lets none of them."""
    calls = []
    monkeypatch.setattr(T, "_given", lambda fn, handle, form, *buffers: calls.append(buffers) and False)
    return calls


def norm_calls():
    p = T.RmsPlan(6, 8)
    x, g, y, c, s, r = torch.zeros(6, 8), torch.zeros(8), torch.zeros(6, 8), torch.zeros(6, 128, dtype=I8), torch.zeros(6), torch.zeros(6)
    f = T.wq8_rms_forward
    return [
        (lambda: f(p, x, g, y=y), 1), (lambda: f(p, x, g, codes=c, scales=s, want_y=False), 1),
        (lambda: f(p, x, g, y=y, codes=c, scales=s, rstd=r, want_codes=True, want_rstd=True), 1), (lambda: f(p, x, g, x, y=y, h=x), 1),
        (lambda: f(p, x, g, y=y, codes=c), 0), (lambda: f(p, x, g, codes=c, want_y=False), 0),  # scales are made
        (lambda: f(p, x, g, codes=c, want_y=False, want_codes=True), 0), (lambda: f(p, x, g, scales=s, y=y), 0),
        (lambda: f(p, x, g), 0), (lambda: f(p, x, g, y=y, want_codes=True), 0), (lambda: f(p, x, g, y=y, want_rstd=True), 0),
        (lambda: f(p, x, g, x, y=y), 0),
    ]


def product_calls():
    p = T.Q8LinearPlan(6, 8, 16, act="silu")
    xq, wq, sx, sw = torch.zeros(6, 128, dtype=I8), torch.zeros(16, 128, dtype=I8), torch.zeros(6), torch.zeros(16)
    y, dx, dw, (zq, sz) = torch.zeros(6, 16), torch.zeros(6, 8), torch.zeros(16, 8), p.empty_z_codes("cpu")
    f, b = T.wq8_q8linear_forward, T.wq8_q8linear_backward
    a = (p, xq, sx, wq, sw)
    return [
        (lambda: f(*a, y=y), 1), (lambda: f(*a, y=y, z=y), 1), (lambda: f(*a, y=y, zq=zq, sz=sz), 1), (lambda: f(*a, y=y, zq=zq), 0),
        (lambda: f(*a, y=y, sz=sz), 0), (lambda: f(*a, y=y, want_z=True), 0), (lambda: f(*a, y=y, zq=zq, sz=sz, want_zq=True), 0),
        (lambda: b(p, y, *a[1:], z=y, dx=dx, dw=dw), 1), (lambda: b(p, y, *a[1:], z=y), 0), (lambda: b(p, y, *a[1:], z=y, dx=dx), 0),
        (lambda: b(p, y, *a[1:], z=y, zq=zq, sz=sz, dx=dx, dw=dw), 0), (lambda: b(p, y, *a[1:], zq=zq, dx=dx, dw=dw), 0),
        (lambda: b(p, y, *a[1:], dx=dx, dw=dw), 0), (lambda: b(p, y, *a[1:], z=y, dx=dx, dw=dw, want_dbias=True), 0),
    ]


@pytest.mark.parametrize("make", [norm_calls, product_calls])
def test_only_calls_that_make_nothing(short, make):
    for i, (call, count) in enumerate(make()):
        short.clear()
        with pytest.raises(ValueError):  # no buffer is on a GPU, on the longer way
            call()
        assert len(short) == count, i


@pytest.mark.gpu
@pytest.mark.parametrize("y_given", [False, True])
def test_scales_are_made_for_given_codes(y_given):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    p = T.RmsPlan(6, 300)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, gamma = torch.randn(6, 300, generator=g, device="cuda"), torch.randn(300, generator=g, device="cuda")
    want = T.wq8_rms_forward(p, x, gamma, want_codes=True)
    kw = dict(y=p.empty_output()) if y_given else dict(want_y=False)
    for stream in (None, torch.cuda.current_stream()):
        codes = torch.full(p.code_shape, 55, dtype=I8, device="cuda")
        y, _, c, s, _ = T.wq8_rms_forward(p, x, gamma, codes=codes, **kw, stream=stream)
        assert c is codes and torch.equal(c, want[2]) and torch.equal(s, want[3])
        assert y is None if not y_given else torch.equal(y, want[0])
