"""ctypes binding of the operators around the convolution (wino_q8_ops.h):
group norm with an activation, and the matrix product with bias, activation
and residual, forward and backward (argument marshalling only).

Every function has the name of the C entry point it calls. Buffers are checked
against the plan before anything reaches the library, ValueError otherwise;
the library's own refusals raise Wq8Error.

A call runs on `stream`, or on the current one; outputs and workspaces that it
makes are allocated as that stream's. Buffers that a caller gives are ordered
and kept by the caller, as with any work on another stream than their own. No
autograd graph is recorded: the backwards are functions of their own, and a
tensor that requires a gradient is refused unless under torch.no_grad(). One that
carries a tangent of forward-mode differentiation is refused: none would come out.
"""
from __future__ import annotations

import ctypes as C

import torch
from torch.autograd import forward_ad

from .binding import _DT, _check, load

ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
LAYOUTS = {"nhwc": 0, "nchw": 1}


class wq8_norm_desc(C.Structure):
    _fields_ = [("N", C.c_int), ("C", C.c_int), ("H", C.c_int), ("W", C.c_int), ("groups", C.c_int),
                ("eps", C.c_float), ("act", C.c_int), ("x_dtype", C.c_int), ("y_dtype", C.c_int),
                ("x_layout", C.c_int), ("y_layout", C.c_int), ("x_stride", C.c_int), ("y_stride", C.c_int)]


class wq8_linear_desc(C.Structure):
    _fields_ = [("rows", C.c_int64), ("Cin", C.c_int), ("Cout", C.c_int), ("act", C.c_int),
                ("x_dtype", C.c_int), ("y_dtype", C.c_int), ("r_layout", C.c_int), ("pixels", C.c_int),
                ("x_stride", C.c_int), ("y_stride", C.c_int), ("r_stride", C.c_int), ("round_dz", C.c_int)]


def _choice(table, key, name):
    if key not in table:
        raise ValueError(f"{name} must be one of {sorted(map(str, table))}, got {key!r}")
    return table[key]


def _desc(cls, *values):
    """The descriptor; ctypes cuts whole numbers to their fields without a word."""
    d = cls(*values)
    for (name, _), v in zip(cls._fields_, values):
        if isinstance(v, int) and getattr(d, name) != v and name != "eps":
            raise ValueError(f"{name} = {v} does not fit its field")
    return d


class _Plan:
    """Owns a plan handle, its workspace sizes and the buffers' forms."""

    _kind = ""

    def _make(self, desc):
        lib = load()
        self._h = None
        h = C.c_void_p()
        _check(getattr(lib, f"wq8_{self._kind}_plan_create")(C.byref(desc), C.byref(h)))
        self._h = h
        f, b = C.c_size_t(), C.c_size_t()
        _check(getattr(lib, f"wq8_{self._kind}_plan_query")(h, C.byref(f), C.byref(b)))
        self.workspace_bytes, self.backward_workspace_bytes = f.value, b.value
        self._forward = getattr(lib, f"wq8_{self._kind}_forward")
        self._backward = getattr(lib, f"wq8_{self._kind}_backward")
        self._destroy = getattr(lib, f"wq8_{self._kind}_plan_destroy")

    def __del__(self):
        # the module's own names may be gone when the interpreter ends
        if getattr(self, "_destroy", None) is not None:
            self._destroy(self._h)
            self._destroy = None

    @property
    def handle(self):
        return self._h

    def empty_workspace(self, device="cuda"):
        return torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device)

    def empty_backward_workspace(self, device="cuda"):
        return torch.empty(self.backward_workspace_bytes, dtype=torch.uint8, device=device)


def _row_strides(shape, stride):
    """Strides of a tensor whose rows (the last dimension) are `stride` elements apart."""
    s = [1]
    step = stride
    for n in reversed(shape[1:-1]):
        s.insert(0, step)
        step *= n
    return (step, *s)


class NormPlan(_Plan):
    """Group norm with an activation over N images of C channels, H x W.

    act: "none", "relu", "silu", "gelu" (erf) or "gelu_tanh". Layouts: "nhwc"
    (tensors [N][H][W][C]; tokens are H = length, W = 1) or "nchw"
    ([N][C][H][W]). x_stride / y_stride: elements between the pixels of an NHWC
    tensor that is a slice of a wider one (0: contiguous)."""

    _kind = "norm"

    def __init__(self, N, C, H, W, groups=32, eps=1e-5, act="none", x_dtype=torch.float32, y_dtype=None,
                 x_layout="nhwc", y_layout=None, x_stride=0, y_stride=0):
        y_dtype = x_dtype if y_dtype is None else y_dtype
        y_layout = x_layout if y_layout is None else y_layout
        self.N, self.C, self.H, self.W, self.groups, self.eps, self.act = N, C, H, W, groups, eps, act
        self.x_dtype, self.y_dtype, self.x_layout, self.y_layout = x_dtype, y_dtype, x_layout, y_layout
        self.x_stride, self.y_stride = int(x_stride), int(y_stride)
        d = _desc(wq8_norm_desc, N, C, H, W, groups, eps, _choice(ACTS, act, "act"), _choice(_DT, x_dtype, "x_dtype"),
                  _choice(_DT, y_dtype, "y_dtype"), _choice(LAYOUTS, x_layout, "x_layout"),
                  _choice(LAYOUTS, y_layout, "y_layout"), self.x_stride, self.y_stride)
        self._make(d)
        self.x_shape = (N, H, W, C) if x_layout == "nhwc" else (N, C, H, W)
        self.y_shape = (N, H, W, C) if y_layout == "nhwc" else (N, C, H, W)
        self.x_strides = _row_strides(self.x_shape, self.x_stride) if self.x_stride else None
        self.y_strides = _row_strides(self.y_shape, self.y_stride) if self.y_stride else None

    def empty_input(self, device="cuda"):
        """A tensor of x's form (for dx)."""
        return _empty(self.x_shape, self.x_stride, self.x_dtype, device)

    def empty_output(self, device="cuda"):
        return _empty(self.y_shape, self.y_stride, self.y_dtype, device)

    def empty_stats(self, device="cuda"):
        """mean and rstd, which the backward needs."""
        return tuple(torch.empty((self.N, self.groups), dtype=torch.float32, device=device) for _ in range(2))


class LinearPlan(_Plan):
    """y = act(x w^T + bias) + residual over `rows` rows (pixels or tokens).

    r_layout "nchw": the residual is [rows / pixels][Cout][pixels], as a
    convolution gives it. x_stride, y_stride, r_stride: elements between the
    rows of tensors that are slices of wider ones (0: contiguous). round_dz: the
    backward of bf16 inputs rounds dz = dy act'(z) to bf16, for half the matrix
    work and 1.4 times the error in dx and dw (False: to 16 bits)."""

    _kind = "linear"

    def __init__(self, rows, Cin, Cout, act="none", x_dtype=torch.float32, y_dtype=None, r_layout="nhwc", pixels=0,
                 x_stride=0, y_stride=0, r_stride=0, round_dz=False):
        y_dtype = x_dtype if y_dtype is None else y_dtype
        self.rows, self.Cin, self.Cout, self.act = rows, Cin, Cout, act
        self.x_dtype, self.y_dtype, self.r_layout, self.pixels = x_dtype, y_dtype, r_layout, pixels
        self.x_stride, self.y_stride, self.r_stride = int(x_stride), int(y_stride), int(r_stride)
        self.round_dz = bool(round_dz)
        d = _desc(wq8_linear_desc, rows, Cin, Cout, _choice(ACTS, act, "act"), _choice(_DT, x_dtype, "x_dtype"),
                  _choice(_DT, y_dtype, "y_dtype"), _choice(LAYOUTS, r_layout, "r_layout"), pixels,
                  self.x_stride, self.y_stride, self.r_stride, self.round_dz)
        self._make(d)
        self.x_shape, self.y_shape, self.w_shape = (rows, Cin), (rows, Cout), (Cout, Cin)
        self.r_shape = (rows // pixels, Cout, pixels) if r_layout == "nchw" else self.y_shape
        self.x_strides = (self.x_stride, 1) if self.x_stride else None
        self.y_strides = (self.y_stride, 1) if self.y_stride else None
        self.r_strides = (self.r_stride, 1) if self.r_stride else None

    def empty_input(self, device="cuda"):
        """A tensor of x's form (for dx)."""
        return _empty(self.x_shape, self.x_stride, self.x_dtype, device)

    def empty_output(self, device="cuda"):
        return _empty(self.y_shape, self.y_stride, self.y_dtype, device)

    def empty_z(self, device="cuda"):
        """The product before its activation, which the backward needs."""
        return torch.empty(self.y_shape, dtype=self.y_dtype, device=device)


def _empty(shape, stride, dtype, device):
    if not stride:
        return torch.empty(shape, dtype=dtype, device=device)
    return torch.empty(shape[:-1] + (stride,), dtype=dtype, device=device)[..., :shape[-1]]


# The stream handle of a device without a Stream object around it, where torch
# offers that: a microsecond less in front of kernels that take five.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class _Args:
    """Checks the buffers of one call: torch tensors of the dtype, shape and
    strides that the plan gives, all on one GPU. The kernels size their
    accesses from the plan, so anything else would be out of bounds."""

    __slots__ = ("stream", "device", "where", "ws", "dual")

    def __init__(self, stream=None):
        self.stream = stream
        self.device = None  # index; -1: not a GPU
        self.where = None   # the first buffer and its name
        self.ws = None      # the workspace, kept until the call is enqueued
        self.dual = forward_ad._current_level >= 0  # whether tensors may carry tangents

    def need(self, t, name, dtype, shape, strides=None):
        """The tensor's address."""
        try:
            if t.dtype != dtype:
                raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
            if t.shape != shape:
                raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
            if strides is None:
                if not t.is_contiguous():
                    raise ValueError(f"{name} must be contiguous")
            elif any(n > 1 and a != b for n, a, b in zip(shape, t.stride(), strides)):
                raise ValueError(f"{name} must have strides {tuple(strides)}, got {tuple(t.stride())}")
            if t.requires_grad and torch.is_grad_enabled():
                raise ValueError(f"{name} requires a gradient, and no graph is recorded here: call this under "
                                 "torch.no_grad() and form gradients with the operator's backward")
            if self.dual and forward_ad.unpack_dual(t).tangent is not None:
                raise ValueError(f"{name} carries a tangent, and no tangents are formed here: give its primal")
            d = t.get_device()
            if d != self.device:
                if self.device is not None:
                    raise ValueError(f"{name} is on {t.device}, {self.where[1]} on {self.where[0].device}")
                self.device = d
                self.where = (t, name)
            return t.data_ptr()
        except AttributeError:
            raise ValueError(f"{name} is required" if t is None else f"{name} must be a torch tensor") from None

    def optional(self, t, name, dtype, shape, strides=None):
        return None if t is None else self.need(t, name, dtype, shape, strides)

    def make(self, fn, *args, **kw):
        """fn(*args, **kw); what it allocates belongs to the call's stream: torch
        hands a freed block out again in the order of the stream it belongs to."""
        if self.stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(self.stream):
            return fn(*args, **kw)

    def workspace(self, t, nbytes):
        """(address, bytes) of a workspace, made here if the caller has none."""
        if nbytes == 0:
            return None, 0
        if t is None:
            t = self.ws = self.make(torch.empty, nbytes, dtype=torch.uint8, device=self.where[0].device)
        if not isinstance(t, torch.Tensor):
            raise ValueError("workspace must be a torch tensor")
        have = t.numel() * t.element_size()
        if have < nbytes:
            raise ValueError(f"workspace holds {have} bytes, needs {nbytes}")
        if not t.is_contiguous():
            raise ValueError("workspace must be contiguous")
        if t.get_device() != self.device:
            raise ValueError(f"workspace is on {t.device}, {self.where[1]} on {self.where[0].device}")
        return t.data_ptr(), have

    def call(self, fn, args):
        """The C call with the buffers' device current, on the call's stream or
        that device's current one."""
        d, stream = self.device, self.stream
        if not self.where[0].is_cuda:
            raise ValueError(f"{self.where[1]} must be on a GPU, got {self.where[0].device}")
        if stream is not None:
            if stream.device.index != d:
                raise ValueError(f"{self.where[1]} is on {self.where[0].device}, the stream on {stream.device}")
            handle = stream.cuda_stream
        else:
            handle = _raw_stream(d) if _raw_stream else torch.cuda.current_stream(d).cuda_stream
        if torch.cuda.current_device() == d:
            st = fn(*args, handle)
        else:
            with torch.cuda.device(d):
                st = fn(*args, handle)
        if st:
            _check(st)


def wq8_norm_forward(plan: NormPlan, x, gamma=None, beta=None, shift=None, y=None, mean=None, rstd=None,
                     want_stats=False, workspace=None, stream=None):
    """y, or (y, mean, rstd) with want_stats."""
    f32, C_ = torch.float32, plan.C
    a = _Args(stream)
    px = a.need(x, "x", plan.x_dtype, plan.x_shape, plan.x_strides)
    ps = a.optional(shift, "shift", f32, (plan.N, C_))
    pg = a.optional(gamma, "gamma", f32, (C_,))
    pb = a.optional(beta, "beta", f32, (C_,))
    if y is None:
        y = a.make(plan.empty_output, x.device)
    py = a.need(y, "y", plan.y_dtype, plan.y_shape, plan.y_strides)
    if want_stats and mean is None:
        mean = a.make(torch.empty, (plan.N, plan.groups), dtype=f32, device=x.device)
    if want_stats and rstd is None:
        rstd = a.make(torch.empty, (plan.N, plan.groups), dtype=f32, device=x.device)
    pm = a.optional(mean, "mean", f32, (plan.N, plan.groups))
    pr = a.optional(rstd, "rstd", f32, (plan.N, plan.groups))
    pw, nw = a.workspace(workspace, plan.workspace_bytes)
    a.call(plan._forward, (plan._h, px, ps, pg, pb, py, pm, pr, pw, nw))
    return (y, mean, rstd) if want_stats else y


def wq8_norm_backward(plan: NormPlan, dy, x, mean, rstd, gamma=None, beta=None, shift=None, dx=None, dgamma=None,
                      dbeta=None, dshift=None, workspace=None, stream=None):
    """(dx, dgamma, dbeta, dshift). Gradients of the parameters that the
    forward was given are made; dgamma and dbeta may be asked for without."""
    f32, C_ = torch.float32, plan.C
    a = _Args(stream)
    pdy = a.need(dy, "dy", plan.y_dtype, plan.y_shape, plan.y_strides)
    px = a.need(x, "x", plan.x_dtype, plan.x_shape, plan.x_strides)
    pm = a.need(mean, "mean", f32, (plan.N, plan.groups))
    pr = a.need(rstd, "rstd", f32, (plan.N, plan.groups))
    pg = a.optional(gamma, "gamma", f32, (C_,))
    pb = a.optional(beta, "beta", f32, (C_,))
    ps = a.optional(shift, "shift", f32, (plan.N, C_))
    if dx is None:
        dx = a.make(plan.empty_input, x.device)
    if dgamma is None and gamma is not None:
        dgamma = a.make(torch.empty, C_, dtype=f32, device=x.device)
    if dbeta is None and beta is not None:
        dbeta = a.make(torch.empty, C_, dtype=f32, device=x.device)
    if dshift is None and shift is not None:
        dshift = a.make(torch.empty, (plan.N, C_), dtype=f32, device=x.device)
    pdx = a.need(dx, "dx", plan.x_dtype, plan.x_shape, plan.x_strides)
    pdg = a.optional(dgamma, "dgamma", f32, (C_,))
    pdb = a.optional(dbeta, "dbeta", f32, (C_,))
    pds = a.optional(dshift, "dshift", f32, (plan.N, C_))
    pw, nw = a.workspace(workspace, plan.backward_workspace_bytes)
    a.call(plan._backward, (plan._h, pdy, px, ps, pg, pb, pm, pr, pdx, pdg, pdb, pds, pw, nw))
    return dx, dgamma, dbeta, dshift


def wq8_linear_forward(plan: LinearPlan, x, w, bias=None, residual=None, y=None, z=None, want_z=False,
                       workspace=None, stream=None):
    """y, or (y, z) with want_z."""
    a = _Args(stream)
    px = a.need(x, "x", plan.x_dtype, plan.x_shape, plan.x_strides)
    pw = a.need(w, "w", plan.x_dtype, plan.w_shape)
    pb = a.optional(bias, "bias", torch.float32, (plan.Cout,))
    pr = a.optional(residual, "residual", plan.y_dtype, plan.r_shape, plan.r_strides)
    if y is None:
        y = a.make(plan.empty_output, x.device)
    if want_z and z is None:
        z = a.make(plan.empty_z, x.device)
    py = a.need(y, "y", plan.y_dtype, plan.y_shape, plan.y_strides)
    pz = a.optional(z, "z", plan.y_dtype, plan.y_shape)
    ws, nw = a.workspace(workspace, plan.workspace_bytes)
    a.call(plan._forward, (plan._h, px, pw, pb, pr, py, pz, ws, nw))
    return (y, z) if want_z else y


def wq8_linear_backward(plan: LinearPlan, dy, x, w, z=None, dx=None, dw=None, dbias=None, want_dx=True, want_dw=True,
                        want_dbias=False, workspace=None, stream=None):
    """(dx, dw, dbias); what is neither given nor wanted is None."""
    a = _Args(stream)
    pdy = a.need(dy, "dy", plan.y_dtype, plan.y_shape, plan.y_strides)
    px = a.need(x, "x", plan.x_dtype, plan.x_shape, plan.x_strides)
    pw = a.need(w, "w", plan.x_dtype, plan.w_shape)
    pz = a.need(z, "z", plan.y_dtype, plan.y_shape) if plan.act != "none" else None
    if dx is None and want_dx:
        dx = a.make(plan.empty_input, x.device)
    if dw is None and want_dw:
        dw = a.make(torch.empty, plan.w_shape, dtype=plan.x_dtype, device=x.device)
    if dbias is None and want_dbias:
        dbias = a.make(torch.empty, plan.Cout, dtype=torch.float32, device=x.device)
    pdx = a.optional(dx, "dx", plan.x_dtype, plan.x_shape, plan.x_strides)
    pdw = a.optional(dw, "dw", plan.x_dtype, plan.w_shape)
    pdb = a.optional(dbias, "dbias", torch.float32, (plan.Cout,))
    ws, nw = a.workspace(workspace, plan.backward_workspace_bytes)
    a.call(plan._backward, (plan._h, pdy, px, pw, pz, pdx, pdw, pdb, ws, nw))
    return dx, dw, dbias
