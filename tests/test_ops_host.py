"""Host-side checks of the group norm and the matrix product: descriptors,
pointers and buffers are refused before anything is launched."""
import ctypes as C
import math

import pytest
import torch

from quantized_convolution_amd import binding as B
from quantized_convolution_amd import ops as O

HAS_GPU = torch.cuda.is_available()
F32, BF = torch.float32, torch.bfloat16


def create(kind, desc):
    h = C.c_void_p()
    st = getattr(B.load(), f"wq8_{kind}_plan_create")(C.byref(desc), C.byref(h))
    assert (st == 0) == bool(h)
    if st == 0:
        getattr(B.load(), f"wq8_{kind}_plan_destroy")(h)
    return st


@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(N=0), 0), (dict(N=-1), -1), (dict(C=0), -1), (dict(H=0), -1), (dict(W=-3), -1),
    (dict(groups=0), -1), (dict(groups=3), -1), (dict(groups=64), 0), (dict(C=7, groups=7), 0),
    (dict(eps=-1e-5), -1), (dict(eps=math.nan), -1), (dict(eps=math.inf), -1), (dict(eps=0.0), 0),
    (dict(act=5), -1), (dict(act=-1), -1), (dict(act=4), 0), (dict(x_dtype=2), -1), (dict(y_dtype=-1), -1),
    (dict(x_layout=2), -1), (dict(y_layout=-1), -1), (dict(x_stride=63), -1), (dict(x_stride=64), 0),
    (dict(x_stride=65, x_layout=1), -1), (dict(y_stride=100), 0), (dict(y_stride=-64), -1),
    (dict(C=1 << 16, H=1 << 8, W=1 << 8), -2), (dict(N=1 << 30, C=64), -2),
])
def test_norm_descriptor(kw, status):
    d = dict(N=2, C=64, H=5, W=7, groups=32, eps=1e-5, act=2, x_dtype=0, y_dtype=0, x_layout=0, y_layout=0, x_stride=0,
             y_stride=0)
    d.update(kw)
    assert create("norm", O.wq8_norm_desc(*d.values())) == status


@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(rows=0), 0), (dict(rows=-1), -1), (dict(Cin=0), -1), (dict(Cout=0), -1), (dict(act=9), -1),
    (dict(x_dtype=3), -1), (dict(y_dtype=2), -1), (dict(r_layout=2), -1), (dict(r_layout=1), -1),
    (dict(r_layout=1, pixels=25), 0), (dict(r_layout=1, pixels=7), -1), (dict(x_stride=39), -1), (dict(x_stride=40), 0),
    (dict(y_stride=20), -1), (dict(r_stride=47), -1), (dict(r_stride=50), 0), (dict(r_stride=50, r_layout=1, pixels=5), -1),
    (dict(rows=1 << 31), -2), (dict(Cin=1 << 22), -2), (dict(x_stride=1 << 22), -2), (dict(rows=(1 << 31) - 2000), 0),
])
def test_linear_descriptor(kw, status):
    d = dict(rows=100, Cin=40, Cout=48, act=1, x_dtype=1, y_dtype=1, r_layout=0, pixels=0, x_stride=0, y_stride=0, r_stride=0)
    d.update(kw)
    assert create("linear", O.wq8_linear_desc(*d.values())) == status


def test_null_arguments():
    lib = B.load()
    for kind in ("norm", "linear"):
        assert getattr(lib, f"wq8_{kind}_plan_create")(None, C.byref(C.c_void_p())) == -1
        assert getattr(lib, f"wq8_{kind}_plan_query")(None, None, None) == -1
        getattr(lib, f"wq8_{kind}_plan_destroy")(None)
    assert lib.wq8_norm_forward(*[None] * 9, 0, None) == -1
    assert lib.wq8_linear_backward(*[None] * 9, 0, None) == -1


@pytest.mark.skipif(HAS_GPU, reason="host-only argument checks; uses fake device pointers")
def test_pointers_are_refused_before_launch():
    lib = B.load()
    p = lambda k: C.c_void_p(0x10000 * (k + 1))  # noqa: E731
    odd = C.c_void_p(0x10004)
    n = O.NormPlan(1, 256, 200, 200, 2, act="silu")
    assert n.workspace_bytes > 0 and n.backward_workspace_bytes > 0
    f = lib.wq8_norm_forward

    def norm(x=p(0), shift=None, gamma=p(1), beta=p(2), y=p(3), mean=None, rstd=None, ws=p(4), nb=n.workspace_bytes):
        return f(n.handle, x, shift, gamma, beta, y, mean, rstd, ws, nb, None)

    assert norm(x=None) == -1 and norm(y=None) == -1 and norm(x=odd) == -5 and norm(gamma=odd) == -5
    assert norm(shift=odd) == -5 and norm(mean=odd) == -5 and norm(y=p(0)) == -1
    assert norm(nb=n.workspace_bytes - 1) == -4 and norm(ws=None) == -1 and norm(ws=odd) == -5
    b = lib.wq8_norm_backward
    wb = n.backward_workspace_bytes
    ok = [p(0), p(1), None, p(2), p(3), p(4), p(5), p(6), p(7), p(8), None, p(9), wb, None]
    for at, bad, want in ((0, None, -1), (1, odd, -5), (5, None, -1), (6, None, -1), (7, None, -1), (7, p(1), -1), (7, p(0), -1),
                          (8, odd, -5), (10, odd, -5), (11, None, -1), (12, wb - 1, -4)):
        assert b(n.handle, *ok[:at], bad, *ok[at + 1:]) == want, at
    lp = O.LinearPlan(64, 4096, 64, act="silu")
    assert lp.workspace_bytes > 0
    ok = [p(0), p(1), p(2), p(3), p(4), None, p(5), lp.workspace_bytes, None]
    for at, bad, want in ((0, None, -1), (1, odd, -5), (2, odd, -5), (3, odd, -5), (4, None, -1), (4, p(0), -1), (4, p(1), -1),
                          (5, p(4), -1), (5, p(3), -1), (5, odd, -5), (6, None, -1), (7, lp.workspace_bytes - 1, -4)):
        assert lib.wq8_linear_forward(lp.handle, *ok[:at], bad, *ok[at + 1:]) == want, at
    wb = lp.backward_workspace_bytes
    ok = [p(0), p(1), p(2), p(3), p(4), p(5), p(6), p(7), wb, None]
    for at, bad, want in ((0, None, -1), (1, None, -1), (2, None, -1), (3, None, -1), (4, p(0), -1), (4, p(5), -1), (5, p(2), -1),
                          (5, odd, -5), (6, odd, -5), (7, None, -1), (8, wb - 1, -4)):
        assert lib.wq8_linear_backward(lp.handle, *ok[:at], bad, *ok[at + 1:]) == want, at


def norm_cases():
    n = O.NormPlan(2, 16, 4, 5, groups=4, y_stride=24)
    x, y, s = torch.zeros(n.x_shape), n.empty_output("cpu"), torch.zeros(2, 4)
    g = torch.zeros(16)
    f, b = O.wq8_norm_forward, O.wq8_norm_backward
    return [
        (lambda: f(n, None, y=y), "x is required"), (lambda: f(n, "x", y=y), "x must be a torch tensor"),
        (lambda: f(n, x.double(), y=y), "x must be"), (lambda: f(n, x[:, :3], y=y), "x must have shape"),
        (lambda: f(n, x.transpose(1, 2).contiguous().transpose(1, 2), y=y), "x must be contiguous"),
        (lambda: f(n, x, g[:8], y=y), "gamma must have shape"), (lambda: f(n, x, g, g.double(), y=y), "beta must be"),
        (lambda: f(n, x, shift=g, y=y), "shift must have shape"),
        (lambda: f(n, x, y=torch.zeros(n.y_shape)), "y must have strides"),
        (lambda: f(n, x, y=y, mean=torch.zeros(2, 3)), "mean must have shape"),
        (lambda: f(n, x, g, g, y=y), "must be on a GPU"),
        (lambda: b(n, y, x, None, s, dx=x), "mean is required"), (lambda: b(n, x, x, s, s, dx=x), "dy must have strides"),
        (lambda: b(n, y, x, s, s, dx=x[:1]), "dx must have shape"),
        (lambda: b(n, y, x, s, s, dx=x, dgamma=g.bfloat16()), "dgamma must be"),
        (lambda: b(n, y, x, s, s, dx=x, workspace=torch.zeros(4, dtype=torch.uint8)), "workspace holds"),
        (lambda: O.NormPlan(2, 16, 4, 5, act="swish"), "act must be one of"),
        (lambda: O.NormPlan(2, 16, 4, 5, x_layout="chwn"), "x_layout must be one of"),
        (lambda: O.NormPlan(2, 16, 4, 5, x_dtype=torch.float16), "x_dtype must be one of"),
    ]


def linear_cases():
    p = O.LinearPlan(6, 8, 16, act="silu", r_layout="nchw", pixels=3)
    x, w, y, r = torch.zeros(6, 8), torch.zeros(16, 8), torch.zeros(6, 16), torch.zeros(2, 16, 3)
    f, b = O.wq8_linear_forward, O.wq8_linear_backward
    return [
        (lambda: f(p, x[:5], w, y=y), "x must have shape"), (lambda: f(p, x, w.T, y=y), "w must have shape"),
        (lambda: f(p, x, w.bfloat16(), y=y), "w must be"), (lambda: f(p, x, w, x, y=y), "bias must have shape"),
        (lambda: f(p, x, w, None, y, y=y), "residual must have shape"),
        (lambda: f(p, x, w, None, r.transpose(1, 2).contiguous().transpose(1, 2), y=y), "residual must be contiguous"),
        (lambda: f(p, x, w, None, r, y=y[:, :8]), "y must have shape"),
        (lambda: f(p, x, w, None, r, y=y, z=y.double()), "z must be"), (lambda: f(p, x, w, None, r, y=y), "must be on a GPU"),
        (lambda: b(p, y, x, w), "z is required"), (lambda: b(p, y, x, w, z=x), "z must have shape"),
        (lambda: b(p, y, x, w, z=y, dx=x, dw=x), "dw must have shape"),
        (lambda: b(p, y, x, w, z=y, dx=x, dw=w, dbias=x), "dbias must have shape"),
        (lambda: b(p, y, x, w, z=y, dx=x, dw=w, workspace=torch.zeros(3, dtype=torch.uint8)), "workspace holds"),
    ]


@pytest.mark.parametrize("make,count", [(norm_cases, 19), (linear_cases, 14)])
def test_buffers_are_refused(make, count):
    cases = make()
    assert len(cases) == count
    for fn, what in cases:
        with pytest.raises(ValueError, match=what):
            fn()


def test_errors_are_named():
    with pytest.raises(B.Wq8Error, match="groups") as e:
        O.NormPlan(1, 10, 2, 2, groups=3)
    assert e.value.status == -1
    with pytest.raises(B.Wq8Error, match="pixels"):
        O.LinearPlan(10, 4, 4, r_layout="nchw", pixels=3)


@pytest.mark.skipif(not HAS_GPU, reason="needs two kinds of device")
def test_mixed_devices_are_refused():
    n = O.NormPlan(2, 16, 4, 5, groups=4)
    with pytest.raises(ValueError, match="gamma is on cpu, x on cuda"):
        O.wq8_norm_forward(n, torch.zeros(n.x_shape, device="cuda"), torch.zeros(16))


@pytest.mark.parametrize("rows,Cin,Cout", [(16, 32, 24), (16384, 100, 3), (16384, 6, 10240), (4000, 640, 2560)])
def test_dz_has_one_form_at_every_size(rows, Cin, Cout):
    """The workspace holds dz of bf16 inputs to 16 bits (4 bytes a value), or rounded where the caller says so (2)."""
    exact, rounded = (O.LinearPlan(rows, Cin, Cout, act="silu", x_dtype=BF, round_dz=r) for r in (False, True))
    values = rows * Cout
    assert exact.backward_workspace_bytes >= 4 * values
    assert 2 * values <= rounded.backward_workspace_bytes
    # dy of x's type without an activation is dz itself
    for r in (False, True):
        assert O.LinearPlan(rows, Cin, Cout, x_dtype=BF, round_dz=r).workspace_bytes == rounded.workspace_bytes
    d = O.wq8_linear_desc(rows, Cin, Cout, 2, 1, 1, 0, 0, 0, 0, 0, 2)
    assert create("linear", d) == -1


class _Allocations:
    """What ops.py allocates in one call: (bytes, made under the call's stream, weak reference)."""

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
    n = O.NormPlan(1, 256, 60, 60, 2, act="silu")
    p = O.LinearPlan(64, 4096, 64, act="silu")
    g, s = torch.zeros(256), torch.zeros(1, 2)
    x, y, z, w = torch.zeros(n.x_shape), torch.zeros(64, 64), torch.zeros(64, 64), torch.zeros(64, 4096)
    t = torch.zeros(64, 4096)
    return [
        (n.workspace_bytes, 4, lambda **kw: O.wq8_norm_forward(n, x, g, g, want_stats=True, **kw)),
        (n.backward_workspace_bytes, 5, lambda **kw: O.wq8_norm_backward(n, x, x, s, s, g, g, shift=torch.zeros(1, 256), **kw)),
        (p.workspace_bytes, 3, lambda **kw: O.wq8_linear_forward(p, t, w, want_z=True, **kw)),
        (p.backward_workspace_bytes, 4, lambda **kw: O.wq8_linear_backward(p, y, t, w, z=z, want_dbias=True, **kw)),
    ]


@pytest.mark.parametrize("which", range(4))
def test_workspace_lives_through_the_call(monkeypatch, which):
    """A workspace made for the caller must not be back with the allocator before
    the kernels are enqueued: another thread could be given the same memory."""
    nbytes, count, run = op_calls()[which]
    a = _Allocations(monkeypatch)
    run()
    assert [n for n, _, _ in a.made].count(nbytes) >= 1 and len(a.made) == count
    assert a.alive_at_call == [True] * count


@pytest.mark.parametrize("which", range(4))
def test_what_a_call_makes_belongs_to_its_stream(monkeypatch, which):
    """Workspaces and outputs made for a call on another stream come from that
    stream's memory: what the current one has freed may still be in use there,
    and what it allocates next must not be this call's workspace."""
    _, count, run = op_calls()[which]
    a = _Allocations(monkeypatch)
    run(stream="another stream")
    assert [inside for _, inside, _ in a.made] == [True] * count
    assert not a.inside


@pytest.mark.parametrize("x_layout,y_layout", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("N,C,H,W,groups,status", [
    (1, 1, 46340, 46341, 1, -2),        # the last block's end would be pixel 2^31
    (1, 1, 1, (1 << 31) - 1, 1, -2), (1, 1, 46340, 46280, 1, 0),
    (1, (1 << 31) - 1, 1, 1, 1, -2), (1, (1 << 31) - 64, 1, 1, 1, -2), (1, 1 << 30, 1, 1, 4, 0),
])
def test_positions_fit_32_bits(N, C, H, W, groups, status, x_layout, y_layout):
    """Pixels and channels are counted in 32 bits, those that a block's last
    steps would reach past the image's end among them."""
    for t in (0, 1):
        d = O.wq8_norm_desc(N, C, H, W, groups, 1e-5, 2, t, t, x_layout, y_layout, 0, 0)
        assert create("norm", d) == status


def test_gradients_are_not_dropped():
    """The operators record no graph: a tensor that asks for one is refused, and taken where none is recorded."""
    n, p = O.NormPlan(2, 16, 4, 5, groups=4), O.LinearPlan(6, 8, 16)
    x, g, s = torch.zeros(n.x_shape), torch.zeros(16), torch.zeros(2, 4)
    t, w, y = torch.zeros(6, 8), torch.zeros(16, 8), torch.zeros(6, 16)
    ask = lambda v: v.clone().requires_grad_()  # noqa: E731
    calls = [(lambda: O.wq8_norm_forward(n, ask(x), y=x), "x"), (lambda: O.wq8_norm_forward(n, x, ask(g), y=x), "gamma"),
             (lambda: O.wq8_norm_forward(n, x, g, ask(g), y=x), "beta"),
             (lambda: O.wq8_norm_forward(n, x, shift=ask(torch.zeros(2, 16)), y=x), "shift"),
             (lambda: O.wq8_norm_backward(n, ask(x), x, s, s, dx=x), "dy"),
             (lambda: O.wq8_linear_forward(p, ask(t), w, y=y), "x"), (lambda: O.wq8_linear_forward(p, t, ask(w), y=y), "w"),
             (lambda: O.wq8_linear_forward(p, t, w, ask(g), y=y), "bias"),
             (lambda: O.wq8_linear_forward(p, t, w, None, ask(y), y=y), "residual"),
             (lambda: O.wq8_linear_backward(p, y, t, ask(w), dx=t, dw=w), "w")]
    for fn, name in calls:
        with pytest.raises(ValueError, match=f"^{name} requires a gradient"):
            fn()
        with torch.no_grad(), pytest.raises(ValueError, match="must be on a GPU"):
            fn()


def test_sizes_are_not_cut_to_32_bits():
    """A size that the descriptor's field does not hold is refused: cut off, the kernels would work on other sizes than the buffers have."""
    for kw in (dict(N=(1 << 32) + 2), dict(C=(1 << 32) + 64), dict(H=1 << 32), dict(groups=(1 << 32) + 4), dict(x_stride=1 << 32),
               dict(y_stride=(1 << 32) + 80)):
        name, = kw
        with pytest.raises(ValueError, match=f"^{name} = "):
            O.NormPlan(**{**dict(N=2, C=64, H=4, W=5, groups=4), **kw})
    for kw in (dict(rows=1 << 64), dict(Cin=(1 << 32) + 8), dict(Cout=-(1 << 32) + 16), dict(pixels=(1 << 32) + 3), dict(r_stride=1 << 32)):
        name, = kw
        with pytest.raises(ValueError, match=f"^{name} = "):
            O.LinearPlan(**{**dict(rows=6, Cin=8, Cout=16), **kw})
