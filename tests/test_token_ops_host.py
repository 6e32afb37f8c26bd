"""Host-side checks of the operators on 8-bit codes: descriptors, pointers and
buffers are refused before anything is launched; and the reference's codes are
what their definition says."""
import ctypes as C
import math

import numpy as np
import pytest
import token_reference as R
import torch

from quantized_convolution_amd import binding as B
from quantized_convolution_amd import ops as O
from quantized_convolution_amd import token_ops as T

HAS_GPU = torch.cuda.is_available()
F32, BF, I8 = torch.float32, torch.bfloat16, torch.int8


def create(kind, desc):
    h = C.c_void_p()
    st = getattr(B.load(), f"wq8_{kind}_plan_create")(C.byref(desc), C.byref(h))
    assert (st == 0) == bool(h)
    if st == 0:
        getattr(B.load(), f"wq8_{kind}_plan_destroy")(h)
    return st


@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(rows=0), 0), (dict(rows=-1), -1), (dict(C=0), -1), (dict(C=1), 0), (dict(group=32), 0), (dict(group=64), 0),
    (dict(group=128), 0), (dict(group=16), -1), (dict(group=-32), -1), (dict(group=256), -1), (dict(x_dtype=2), -1),
    (dict(x_stride=39), -1), (dict(x_stride=41), 0), (dict(x_stride=-1), -1), (dict(rows=1 << 31), -2), (dict(C=1 << 20), -2),
    (dict(C=(1 << 20) - 1), 0), (dict(rows=(1 << 31) - 2000, C=1 << 19), -2),
])
def test_quant_descriptor(kw, status):
    d = dict(rows=100, C=40, group=0, x_dtype=1, x_stride=0)
    d.update(kw)
    assert create("quant", T.wq8_quant_desc(*d.values())) == status


@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(rows=0), 0), (dict(rows=-1), -1), (dict(C=0), -1), (dict(eps=-1e-5), -1), (dict(eps=math.nan), -1),
    (dict(eps=math.inf), -1), (dict(eps=0.0), 0), (dict(x_dtype=2), -1), (dict(y_dtype=-1), -1), (dict(x_stride=39), -1),
    (dict(x_stride=50), 0), (dict(y_stride=39), -1), (dict(y_stride=40), 0), (dict(rows=1 << 31), -2), (dict(C=1 << 20), -2),
])
def test_rms_descriptor(kw, status):
    d = dict(rows=100, C=40, eps=1e-6, x_dtype=1, y_dtype=0, x_stride=0, y_stride=0)
    d.update(kw)
    assert create("rms", T.wq8_rms_desc(*d.values())) == status


@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(rows=0), 0), (dict(rows=-1), -1), (dict(Cin=0), -1), (dict(Cout=0), -1), (dict(act=5), -1), (dict(act=-1), -1),
    (dict(x_dtype=3), -1), (dict(y_dtype=2), -1), (dict(r_layout=2), -1), (dict(r_layout=1), -1), (dict(r_layout=1, pixels=25), 0),
    (dict(r_layout=1, pixels=7), -1), (dict(x_stride=39), -1), (dict(y_stride=20), -1), (dict(r_stride=47), -1),
    (dict(r_stride=50), 0), (dict(r_stride=50, r_layout=1, pixels=5), -1), (dict(rows=1 << 24), -2), (dict(Cin=1 << 20), -2),
    (dict(Cout=1 << 20), -2), (dict(rows=(1 << 24) - 1), 0), (dict(rows=1, Cin=(1 << 20) - 1), 0),
])
def test_product_descriptor(kw, status):
    d = dict(rows=100, Cin=40, Cout=48, act=1, x_dtype=1, y_dtype=1, r_layout=0, pixels=0, x_stride=0, y_stride=0, r_stride=0)
    d.update(kw)
    assert create("q8linear", T.wq8_q8linear_desc(*d.values())) == status


def test_null_arguments():
    lib = B.load()
    for kind in ("quant", "rms", "q8linear"):
        assert getattr(lib, f"wq8_{kind}_plan_create")(None, C.byref(C.c_void_p())) == -1
        getattr(lib, f"wq8_{kind}_plan_destroy")(None)
    for kind in ("rms", "q8linear"):
        assert getattr(lib, f"wq8_{kind}_plan_query")(None, None, None) == -1
    assert lib.wq8_quant_pack(*[None] * 5) == -1 and lib.wq8_quant_unpack(*[None] * 5) == -1
    assert lib.wq8_rms_forward(*[None] * 10, 0, None) == -1 and lib.wq8_rms_backward(*[None] * 9, 0, None) == -1
    assert lib.wq8_q8linear_forward(*[None] * 12, 0, None) == -1 and lib.wq8_q8linear_backward(*[None] * 13, 0, None) == -1


@pytest.mark.skipif(HAS_GPU, reason="host-only argument checks; uses fake device pointers")
def test_pointers_are_refused_before_launch():
    lib = B.load()
    p = lambda k: C.c_void_p(0x10000 * (k + 1))  # noqa: E731
    odd = C.c_void_p(0x10004)

    def refused(f, h, ok, cases):
        for changes, want in cases:
            args = list(ok)
            for at, bad in changes.items():
                args[at] = bad
            assert f(h, *args) == want, changes

    n = T.QuantPlan(10, 100)
    refused(lib.wq8_quant_pack, n.handle, [p(0), p(1), p(2), None],
            [({0: None}, -1), ({1: None}, -1), ({2: None}, -1), ({0: odd}, -5), ({1: odd}, -5), ({2: odd}, -5), ({1: p(0)}, -1),
             ({2: p(1)}, -1), ({2: p(0)}, -1)])
    refused(lib.wq8_quant_unpack, n.handle, [p(0), p(1), p(2), None],
            [({0: None}, -1), ({1: odd}, -5), ({2: None}, -1), ({2: p(0)}, -1), ({2: p(1)}, -1)])
    m = T.RmsPlan(10, 100)
    assert m.workspace_bytes == 0 and m.backward_workspace_bytes > 0
    # x residual gamma h y codes scales rstd workspace bytes stream
    ok = [p(0), p(1), p(2), p(3), p(4), p(5), p(6), p(7), None, 0, None]
    refused(lib.wq8_rms_forward, m.handle, ok,
            [({0: None}, -1), ({1: odd}, -5), ({2: odd}, -5), ({3: odd}, -5), ({4: odd}, -5), ({5: odd}, -5), ({6: odd}, -5),
             ({7: odd}, -5), ({4: None, 5: None, 6: None}, -1), ({5: None}, -1), ({6: None}, -1), ({1: None}, -1),
             ({4: p(0)}, -1), ({4: p(1)}, -1), ({4: p(3)}, -1), ({5: p(0)}, -1), ({3: p(5)}, -1), ({3: p(2)}, -1), ({7: p(6)}, -1),
             ({7: p(2)}, -1)])
    wb = m.backward_workspace_bytes
    # dy h rstd gamma dh dx dgamma workspace
    ok = [p(0), p(1), p(2), p(3), p(4), p(5), p(6), p(7), wb, None]
    refused(lib.wq8_rms_backward, m.handle, ok,
            [({0: None}, -1), ({1: None}, -1), ({2: None}, -1), ({3: odd}, -5), ({4: odd}, -5), ({5: None}, -1), ({5: p(0)}, -1),
             ({5: p(1)}, -1), ({6: p(5)}, -1), ({6: p(3)}, -1), ({6: odd}, -5), ({7: None}, -1), ({8: wb - 1}, -4), ({7: odd}, -5)])
    q = T.Q8LinearPlan(200, 70000, 64, act="silu")
    assert q.workspace_bytes > 0
    # xq sx wq sw bias residual y z zq sz workspace
    ok = [p(0), p(1), p(2), p(3), p(4), p(5), p(6), p(7), p(8), p(9), p(10), q.workspace_bytes, None]
    refused(lib.wq8_q8linear_forward, q.handle, ok,
            [({0: None}, -1), ({1: None}, -1), ({2: None}, -1), ({3: None}, -1), ({4: odd}, -5), ({5: odd}, -5), ({6: None}, -1),
             ({6: p(0)}, -1), ({6: p(2)}, -1), ({7: odd}, -5), ({7: p(6)}, -1), ({7: p(5)}, -1), ({8: None}, -1), ({9: None}, -1),
             ({8: p(2)}, -1), ({9: p(8)}, -1), ({8: odd}, -5), ({9: odd}, -5), ({10: None}, -1), ({10: odd}, -5),
             ({11: q.workspace_bytes - 1}, -4)])
    planar = T.Q8LinearPlan(200, 100, 64, r_layout="nchw", pixels=50)
    refused(lib.wq8_q8linear_forward, planar.handle, ok, [({6: p(5)}, -1)])
    wide = T.Q8LinearPlan(200, 100, 64, r_stride=70)
    refused(lib.wq8_q8linear_forward, wide.handle, ok, [({6: p(5)}, -1)])
    wb = q.backward_workspace_bytes
    # dy xq sx wq sw z zq sz dx dw dbias workspace
    ok = [p(0), p(1), p(2), p(3), p(4), p(5), None, None, p(8), p(9), p(10), p(11), wb, None]
    refused(lib.wq8_q8linear_backward, q.handle, ok,
            [({0: None}, -1), ({1: None}, -1), ({2: None}, -1), ({3: None}, -1), ({4: None}, -1), ({5: None}, -1),
             ({6: p(6), 7: p(7)}, -1), ({5: None, 6: p(6)}, -1), ({5: odd}, -5), ({8: p(0)}, -1), ({8: p(9)}, -1), ({9: p(1)}, -1),
             ({10: p(9)}, -1), ({9: odd}, -5), ({10: odd}, -5), ({11: None}, -1), ({12: wb - 1}, -4)])


def quant_cases():
    p = T.QuantPlan(6, 40, group=32, x_stride=44)
    x, (c, s) = p.empty_input("cpu"), p.empty_codes("cpu")
    f, b = T.wq8_quant_pack, T.wq8_quant_unpack
    return [
        (lambda: f(p, None), "x is required"), (lambda: f(p, torch.zeros(6, 40), c, s), "x must have strides"),
        (lambda: f(p, x.double(), c, s), "x must be"), (lambda: f(p, x, c[:5], s), "codes must have shape"),
        (lambda: f(p, x, c[:, :64], s), "codes must have shape"), (lambda: f(p, x, c, s[:, 0]), "scales must have shape"),
        (lambda: f(p, x, c.float(), s), "codes must be"), (lambda: f(p, x, c, s), "must be on a GPU"),
        (lambda: b(p, c, s[:5], x), "scales must have shape"), (lambda: b(p, c.T, s, x), "codes must have shape"),
        (lambda: b(p, c, s, torch.zeros(6, 40)), "x must have strides"),
        (lambda: T.QuantPlan(6, 40, x_dtype=torch.float16), "x_dtype must be one of"),
    ]


def rms_cases():
    p = T.RmsPlan(6, 40, y_dtype=BF, y_stride=48)
    x, y, (c, s), g = p.empty_input("cpu"), p.empty_output("cpu"), p.empty_codes("cpu"), torch.zeros(40)
    r = torch.zeros(6)
    f, b = T.wq8_rms_forward, T.wq8_rms_backward
    return [
        (lambda: f(p, x[:5], y=y), "x must have shape"), (lambda: f(p, x, g[:8], y=y), "gamma must have shape"),
        (lambda: f(p, x, g, x.bfloat16(), y=y), "residual must be"), (lambda: f(p, x, g, y=x), "y must be"),
        (lambda: f(p, x, g, y=torch.zeros(6, 40, dtype=BF)), "y must have strides"),
        (lambda: f(p, x, g, x, y=y, h=x[:, :8]), "h must have shape"), (lambda: f(p, x, y=y, codes=c[:, :40]), "codes must have shape"),
        (lambda: f(p, x, y=y, codes=c, scales=s[:3]), "scales must have shape"), (lambda: f(p, x, y=y, rstd=g), "rstd must have shape"),
        (lambda: f(p, x, g, y=y), "must be on a GPU"), (lambda: b(p, y, x, None, dx=x), "rstd is required"),
        (lambda: b(p, x, x, r, dx=x), "dy must be"), (lambda: b(p, y, x, r, dh=y, dx=x), "dh must be"),
        (lambda: b(p, y, x, r, dx=x[:2]), "dx must have shape"), (lambda: b(p, y, x, r, g, dx=x, dgamma=r), "dgamma must have shape"),
        (lambda: b(p, y, x, r, g, dx=x, dgamma=g, workspace=torch.zeros(4, dtype=torch.uint8)), "workspace holds"),
    ]


def product_cases():
    p = T.Q8LinearPlan(6, 8, 16, act="silu", r_layout="nchw", pixels=3)
    xq, sx, wq, sw = torch.zeros(6, 128, dtype=I8), torch.zeros(6), torch.zeros(16, 128, dtype=I8), torch.zeros(16)
    y, r, x, w = torch.zeros(6, 16), torch.zeros(2, 16, 3), torch.zeros(6, 8), torch.zeros(16, 8)
    zq, sz = p.empty_z_codes("cpu")
    f, b = T.wq8_q8linear_forward, T.wq8_q8linear_backward
    return [
        (lambda: f(p, xq[:, :8], sx, wq, sw, y=y), "xq must have shape"), (lambda: f(p, xq.float(), sx, wq, sw, y=y), "xq must be"),
        (lambda: f(p, xq, sw, wq, sw, y=y), "sx must have shape"), (lambda: f(p, xq, sx, xq, sw, y=y), "wq must have shape"),
        (lambda: f(p, xq, sx, wq, sx, y=y), "sw must have shape"), (lambda: f(p, xq, sx, wq, sw, sx, y=y), "bias must have shape"),
        (lambda: f(p, xq, sx, wq, sw, None, y, y=y), "residual must have shape"),
        (lambda: f(p, xq, sx, wq, sw, None, r, y=y[:, :8]), "y must have shape"),
        (lambda: f(p, xq, sx, wq, sw, None, r, y=y, z=y.double()), "z must be"),
        (lambda: f(p, xq, sx, wq, sw, None, r, y=y, zq=xq[:3]), "zq must have shape"),
        (lambda: f(p, xq, sx, wq, sw, None, r, y=y, zq=zq, sz=sx), "sz must have shape"),
        (lambda: f(p, xq, sx, wq, sw, None, r, y=y), "must be on a GPU"), (lambda: b(p, y, xq, sx, wq, sw), "z is required"),
        (lambda: b(p, y, xq, sx, wq, sw, z=x), "z must have shape"), (lambda: b(p, y, xq, sx, wq, sw, z=y, zq=zq), "one of the two"),
        (lambda: b(p, y, xq, sx, wq, sw, zq=zq), "sz is required"), (lambda: b(p, x, xq, sx, wq, sw, z=y), "dy must have shape"),
        (lambda: b(p, y, xq, sx, wq, sw, z=y, dx=x, dw=x), "dw must have shape"),
        (lambda: b(p, y, xq, sx, wq, sw, z=y, dx=x, dw=w, dbias=sx), "dbias must have shape"),
        (lambda: b(p, y, xq, sx, wq, sw, z=y, dx=x, dw=w, workspace=torch.zeros(3, dtype=torch.uint8)), "workspace holds"),
        (lambda: T.Q8LinearPlan(6, 8, 16, act="swish"), "act must be one of"),
    ]


@pytest.mark.parametrize("make,count", [(quant_cases, 12), (rms_cases, 16), (product_cases, 21)])
def test_buffers_are_refused(make, count):
    cases = make()
    assert len(cases) == count
    for fn, what in cases:
        with pytest.raises(ValueError, match=what):
            fn()


def test_errors_are_named():
    with pytest.raises(B.Wq8Error, match="group is") as e:
        T.QuantPlan(1, 10, group=5)
    assert e.value.status == -1
    with pytest.raises(B.Wq8Error, match="eps"):
        T.RmsPlan(1, 10, eps=-1.0)
    with pytest.raises(B.Wq8Error, match="pixels"):
        T.Q8LinearPlan(10, 4, 4, r_layout="nchw", pixels=3)


def test_sizes_are_not_cut_to_32_bits():
    for cls, base, kws in ((T.QuantPlan, dict(rows=6, C=8), (dict(C=(1 << 32) + 8), dict(group=(1 << 32) + 32), dict(x_stride=1 << 32))),
                           (T.RmsPlan, dict(rows=6, C=8), (dict(C=(1 << 32) + 8), dict(rows=1 << 64), dict(y_stride=(1 << 32) + 8))),
                           (T.Q8LinearPlan, dict(rows=6, Cin=8, Cout=16),
                            (dict(Cin=(1 << 32) + 8), dict(Cout=-(1 << 32) + 16), dict(pixels=(1 << 32) + 3), dict(r_stride=1 << 32)))):
        for kw in kws:
            name, = kw
            with pytest.raises(ValueError, match=f"^{name} = "):
                cls(**{**base, **kw})


def test_gradients_are_not_dropped():
    """The operators record no graph: a tensor that asks for one is refused, and taken where none is recorded."""
    n, m, p = T.QuantPlan(6, 8), T.RmsPlan(6, 8), T.Q8LinearPlan(6, 8, 16)
    x, g, y, s = torch.zeros(6, 8), torch.zeros(8), torch.zeros(6, 16), torch.zeros(6)
    xq, wq, sw = torch.zeros(6, 128, dtype=I8), torch.zeros(16, 128, dtype=I8), torch.zeros(16)
    ask = lambda v: v.clone().requires_grad_()  # noqa: E731
    calls = [(lambda: T.wq8_quant_pack(n, ask(x), xq, s), "x"), (lambda: T.wq8_rms_forward(m, ask(x), y=x), "x"),
             (lambda: T.wq8_rms_forward(m, x, ask(g), y=x), "gamma"), (lambda: T.wq8_rms_forward(m, x, g, ask(x), y=x, h=x), "residual"),
             (lambda: T.wq8_rms_backward(m, ask(x), x, s, dx=x), "dy"), (lambda: T.wq8_rms_backward(m, x, x, s, dh=ask(x), dx=x), "dh"),
             (lambda: T.wq8_q8linear_forward(p, xq, ask(s), wq, sw, y=y), "sx"),
             (lambda: T.wq8_q8linear_forward(p, xq, s, wq, sw, ask(sw), y=y), "bias"),
             (lambda: T.wq8_q8linear_forward(p, xq, s, wq, sw, None, ask(y), y=y), "residual"),
             (lambda: T.wq8_q8linear_backward(p, ask(y), xq, s, wq, sw, dx=x, dw=torch.zeros(16, 8)), "dy")]
    for fn, name in calls:
        with pytest.raises(ValueError, match=f"^{name} requires a gradient"):
            fn()
        with torch.no_grad(), pytest.raises(ValueError, match="must be on a GPU"):
            fn()


class _Allocations:
    """What a call allocates: (bytes, made under the call's stream, weak reference)."""

    def __init__(self, monkeypatch):
        import contextlib
        import weakref

        self.made, self.inside, self.alive_at_call = [], [], None
        real = torch.empty

        def empty(*args, **kw):
            t = real(*args, **{**kw, "device": "cpu"})
            self.made.append((t.numel() * t.element_size(), bool(self.inside), weakref.ref(t)))
            return t

        @contextlib.contextmanager
        def stream(s):
            if s is not None:
                self.inside.append(s)
            yield
            if s is not None:
                self.inside.pop()

        def call(args, fn, pointers, stream=None):
            self.alive_at_call = [ref() is not None for _, _, ref in self.made]

        monkeypatch.setattr(torch, "empty", empty)
        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(O._Args, "call", call)


def op_calls():
    n, m, p = T.QuantPlan(6, 8), T.RmsPlan(600, 8), T.Q8LinearPlan(200, 70000, 64, act="silu")
    x, g = torch.zeros(600, 8), torch.zeros(8)
    xq, wq = torch.zeros(200, 70016, dtype=I8), torch.zeros(64, 70016, dtype=I8)
    sx, sw, y = torch.zeros(200), torch.zeros(64), torch.zeros(200, 64)
    c, s = torch.zeros(6, 128, dtype=I8), torch.zeros(6)
    return [
        (None, 2, lambda **kw: T.wq8_quant_pack(n, x[:6], **kw)), (None, 1, lambda **kw: T.wq8_quant_unpack(n, c, s, **kw)),
        (None, 5, lambda **kw: T.wq8_rms_forward(m, x, g, x, want_codes=True, want_rstd=True, **kw)),
        (m.backward_workspace_bytes, 3, lambda **kw: T.wq8_rms_backward(m, x, x, x[:, 0].contiguous(), g, **kw)),
        (p.workspace_bytes, 5, lambda **kw: T.wq8_q8linear_forward(p, xq, sx, wq, sw, want_z=True, want_zq=True, **kw)),
        (p.backward_workspace_bytes, 4, lambda **kw: T.wq8_q8linear_backward(p, y, xq, sx, wq, sw, z=y, want_dbias=True, **kw)),
    ]


@pytest.mark.parametrize("which", range(6))
def test_what_a_call_makes(monkeypatch, which):
    """It lives until the kernels are enqueued, and is the call's stream's."""
    nbytes, count, run = op_calls()[which]
    a = _Allocations(monkeypatch)
    run()
    assert len(a.made) == count and a.alive_at_call == [True] * count
    assert nbytes is None or [n for n, _, _ in a.made].count(nbytes) >= 1
    a.made.clear()
    run(stream="another stream")
    assert [inside for _, inside, _ in a.made] == [True] * count and not a.inside


# ------------------------------------------------------------------ the reference
def test_reference_codes_are_nearest():
    """In 64 bits: every code within half a step and its roundings of its value, the largest 127 exactly."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(50, 301, generator=g) * torch.logspace(-30, 30, 50)[:, None]
    for group in (0, 32, 128):
        codes, scales = R.codes_of(x.numpy(), group)
        assert codes.shape == (50, 384) and bool((codes[:, 301:] == 0).all()) and int(codes.min()) >= -127
        v = R.values(codes, scales, 301, group)
        step = scales.double()[:, None] if not group else scales.double().repeat_interleave(group, 1)[:, :301]
        assert bool(((v - x.double()).abs() <= step * (0.5 + 127 * 4 * R.U)).all())
        n = group or 301
        for j in range(0, 301, n):
            assert bool((codes[:, j:j + n].abs().amax(1) == 127).all())


def test_reference_gradients_are_those_of_the_formulas():
    g = torch.Generator().manual_seed(2)
    h, gm, dy = (torch.randn(s, generator=g).double() for s in ((5, 17), (17,), (5, 17)))
    a, b = h.clone().requires_grad_(), gm.clone().requires_grad_()
    y = a / torch.sqrt(a.square().mean(1, keepdim=True) + 1e-6) * b
    want = torch.autograd.grad(y, (a, b), dy)
    ref = R.Rms(h, 1e-6, gm)
    got = ref.backward(dy, ref.rstd, None, F32)
    torch.testing.assert_close(got["dx"][0], want[0], rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(got["dgamma"][0], want[1], rtol=1e-12, atol=1e-12)
    xq, sx = R.codes_of(torch.randn(6, 9, generator=g).numpy())
    wq, sw = R.codes_of(torch.randn(4, 9, generator=g).numpy())
    x, w = R.values(xq, sx, 9).requires_grad_(), R.values(wq, sw, 9).requires_grad_()
    z = x @ w.T
    d = torch.randn(6, 4, generator=g).double()
    want = torch.autograd.grad(R.act(z, "gelu"), (x, w), d)
    got = R.backward(d, xq, sx, wq, sw, 9, F32, "gelu", z.detach())
    torch.testing.assert_close(got["dx"][0], want[0], rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(got["dw"][0], want[1], rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(R.product(xq, sx, wq, sw, 9).numpy(), z.detach().numpy(), rtol=1e-6, atol=1e-6)
