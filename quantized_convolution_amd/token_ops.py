"""ctypes binding of the operators on 8-bit codes (wino_q8_tokens.h): packing of
rows, the root-mean-square norm with an output in codes, and the matrix product
of codes with its backward (argument marshalling only).

Checks, streams, workspaces and errors are those of ops.py: buffers are checked
against the plan before anything reaches the library, ValueError otherwise; the
library's own refusals raise Wq8Error; no autograd graph is recorded.

A tensor held in 8 bits is a pair (codes, scales): int8 [rows][code_stride], rows
in whole lines of 128 bytes with zeros behind the last column, and f32 scales,
[rows], or [rows][groups] where groups of columns have one each.
"""
from __future__ import annotations

import ctypes as C
import warnings

import torch

from .binding import _DT, _check, load
from .ops import ACTS, LAYOUTS, _Args, _choice, _desc, _empty, _Plan, _raw_stream

Z_GROUP = 32  # columns that share a scale where a product's z is kept in codes


class wq8_quant_desc(C.Structure):
    _fields_ = [("rows", C.c_int64), ("C", C.c_int), ("group", C.c_int), ("x_dtype", C.c_int), ("x_stride", C.c_int)]


class wq8_rms_desc(C.Structure):
    _fields_ = [("rows", C.c_int64), ("C", C.c_int), ("eps", C.c_float), ("x_dtype", C.c_int), ("y_dtype", C.c_int),
                ("x_stride", C.c_int), ("y_stride", C.c_int)]


class wq8_q8linear_desc(C.Structure):
    _fields_ = [("rows", C.c_int64), ("Cin", C.c_int), ("Cout", C.c_int), ("act", C.c_int), ("x_dtype", C.c_int),
                ("y_dtype", C.c_int), ("r_layout", C.c_int), ("pixels", C.c_int), ("x_stride", C.c_int), ("y_stride", C.c_int),
                ("r_stride", C.c_int), ("round_dz", C.c_int)]


def code_stride(columns):
    """Bytes of a row of codes: whole lines of 128."""
    return (columns + 127) // 128 * 128


I8, F32 = torch.int8, torch.float32


def _given(fn, handle, form, *buffers):
    """Makes the call on the current stream if every buffer is given and as the
    plan says, all on the current GPU. Else nothing is done: the checks that
    follow name what is wrong, or make what is missing."""
    if form is None:
        return False
    got = _addresses(form, *buffers)
    if got is None or got[0] != torch._C._cuda_getDevice():
        return False
    st = fn(handle, *got[1:], _raw_stream(got[0]))
    if st:
        _check(st)
    return True


_addresses = _form = None  # the module's functions; False where it cannot be loaded


def _load_buffers():
    """The CPython module that is built beside the library. Without it every call
    takes the longer way through the checks."""
    global _addresses, _form
    try:
        from ._wq8_buffers import addresses as _addresses, form as _form
    except ImportError as e:
        _addresses = _form = False
        warnings.warn(f"_wq8_buffers cannot be loaded ({e}): calls whose buffers are all given take some microseconds more. Build it "
                      "again with `python -c 'import __graft_entry__ as g; g.build()'`", RuntimeWarning, stacklevel=4)


def _forms(*entries):
    """The form of a call's buffers, for _given()."""
    if _form is None:
        _load_buffers()
    return _form(tuple(e if isinstance(e, int) else (e[0], tuple(e[1]), e[2], e[3]) for e in entries)) \
        if _form and _raw_stream else None


class QuantPlan(_Plan):
    """Rows of C values to 8-bit codes and back. group: columns that share a
    scale, 32, 64 or 128, or 0 for one scale a row (what products take).
    x_stride: elements between the rows of a tensor that is a slice of a wider
    one (0: contiguous)."""

    _kind = "quant"

    def __init__(self, rows, C, group=0, x_dtype=torch.float32, x_stride=0):
        self.rows, self.C, self.group, self.x_dtype, self.x_stride = rows, C, group, x_dtype, int(x_stride)
        self._make(_desc(wq8_quant_desc, rows, C, group, _choice(_DT, x_dtype, "x_dtype"), self.x_stride))
        self.x_shape, self.x_strides = (rows, C), (self.x_stride, 1) if self.x_stride else None
        self.code_shape = (rows, code_stride(C))
        self.scale_shape = (rows, -(-C // group)) if group else (rows,)
        x = (x_dtype, self.x_shape, self.x_strides, True)
        codes = (I8, self.code_shape, None, True), (F32, self.scale_shape, None, True)
        self._pack_form, self._unpack_form = _forms(x, *codes), _forms(*codes, x)

    def _make(self, desc):
        lib = load()
        self._h = None
        h = C.c_void_p()
        _check(lib.wq8_quant_plan_create(C.byref(desc), C.byref(h)))
        self._h = h
        self._pack, self._unpack, self._destroy = lib.wq8_quant_pack, lib.wq8_quant_unpack, lib.wq8_quant_plan_destroy
        self.workspace_bytes = self.backward_workspace_bytes = 0  # it needs none

    def empty_input(self, device="cuda"):
        """A tensor of x's form."""
        return _empty(self.x_shape, self.x_stride, self.x_dtype, device)

    def empty_codes(self, device="cuda"):
        """(codes, scales)."""
        return _empty_codes(self.code_shape, self.scale_shape, device)


class RmsPlan(_Plan):
    """Root-mean-square norm over rows of C values, y = h rstd gamma, of the
    stream h = x + residual. x_stride: elements between the rows of x, residual,
    h, dh and dx, y_stride: of y and dy, where they are slices of wider tensors
    (0: contiguous)."""

    _kind = "rms"

    def __init__(self, rows, C, eps=1e-6, x_dtype=torch.float32, y_dtype=None, x_stride=0, y_stride=0):
        y_dtype = x_dtype if y_dtype is None else y_dtype
        self.rows, self.C, self.eps, self.x_dtype, self.y_dtype = rows, C, eps, x_dtype, y_dtype
        self.x_stride, self.y_stride = int(x_stride), int(y_stride)
        self._make(_desc(wq8_rms_desc, rows, C, eps, _choice(_DT, x_dtype, "x_dtype"), _choice(_DT, y_dtype, "y_dtype"),
                         self.x_stride, self.y_stride))
        self.x_shape = self.y_shape = (rows, C)
        self.x_strides = (self.x_stride, 1) if self.x_stride else None
        self.y_strides = (self.y_stride, 1) if self.y_stride else None
        self.code_shape, self.scale_shape = (rows, code_stride(C)), (rows,)
        x, y = (lambda r: (x_dtype, self.x_shape, self.x_strides, r)), (lambda r: (y_dtype, self.y_shape, self.y_strides, r))
        row, column = (lambda r: (F32, (rows,), None, r)), (F32, (C,), None, False)
        self._forward_form = _forms(x(True), x(False), column, x(False), y(False), (I8, self.code_shape, None, False), row(False),
                                    row(False), self.workspace_bytes)
        self._backward_form = _forms(y(True), x(True), row(True), column, x(False), x(True), column, self.backward_workspace_bytes)

    def empty_input(self, device="cuda"):
        """A tensor of x's form (for h and dx)."""
        return _empty(self.x_shape, self.x_stride, self.x_dtype, device)

    def empty_output(self, device="cuda"):
        return _empty(self.y_shape, self.y_stride, self.y_dtype, device)

    def empty_codes(self, device="cuda"):
        """(codes, scales)."""
        return _empty_codes(self.code_shape, self.scale_shape, device)

    def empty_rstd(self, device="cuda"):
        """What the backward needs."""
        return torch.empty(self.rows, dtype=torch.float32, device=device)


class Q8LinearPlan(_Plan):
    """y = act(x^ w^^T + bias) + residual, where x^ [rows][Cin] and w^ [Cout][Cin] are
    held in codes with a scale for each row (`QuantPlan` of group 0 makes both).

    x_dtype: of the gradients dx and dw; y_dtype: of y, z, residual and dy.
    r_layout "nchw": the residual is [rows / pixels][Cout][pixels], as a
    convolution gives it. x_stride (dx), y_stride, r_stride: elements between the
    rows of tensors that are slices of wider ones (0: contiguous). round_dz: a
    backward to bf16 holds dz sw and dz sx in 16 bits of the largest of their row or
    column, for half the matrix work. Where one token's gradient is some hundred times
    the others', what these give to dw loses more than bf16's own rounding, and so
    for a loud channel in dx (False: in 32 bits)."""

    _kind = "q8linear"

    def __init__(self, rows, Cin, Cout, act="none", x_dtype=torch.float32, y_dtype=None, r_layout="nhwc", pixels=0, x_stride=0,
                 y_stride=0, r_stride=0, round_dz=False):
        y_dtype = x_dtype if y_dtype is None else y_dtype
        self.rows, self.Cin, self.Cout, self.act = rows, Cin, Cout, act
        self.x_dtype, self.y_dtype, self.r_layout, self.pixels = x_dtype, y_dtype, r_layout, pixels
        self.x_stride, self.y_stride, self.r_stride = int(x_stride), int(y_stride), int(r_stride)
        self.round_dz = bool(round_dz)
        self._make(_desc(wq8_q8linear_desc, rows, Cin, Cout, _choice(ACTS, act, "act"), _choice(_DT, x_dtype, "x_dtype"),
                         _choice(_DT, y_dtype, "y_dtype"), _choice(LAYOUTS, r_layout, "r_layout"), pixels, self.x_stride,
                         self.y_stride, self.r_stride, self.round_dz))
        self.x_shape, self.y_shape, self.w_shape = (rows, Cin), (rows, Cout), (Cout, Cin)
        self.r_shape = (rows // pixels, Cout, pixels) if r_layout == "nchw" else self.y_shape
        self.x_strides = (self.x_stride, 1) if self.x_stride else None
        self.y_strides = (self.y_stride, 1) if self.y_stride else None
        self.r_strides = (self.r_stride, 1) if self.r_stride else None
        self.xq_shape, self.wq_shape = (rows, code_stride(Cin)), (Cout, code_stride(Cin))
        self.zq_shape, self.sz_shape = (rows, code_stride(Cout)), (rows, -(-Cout // Z_GROUP))
        y = (y_dtype, self.y_shape, self.y_strides, True)
        codes = ((I8, self.xq_shape, None, True), (F32, (rows,), None, True), (I8, self.wq_shape, None, True),
                 (F32, (Cout,), None, True))
        column, z = (F32, (Cout,), None, False), (y_dtype, self.y_shape, None, False)
        zq = (I8, self.zq_shape, None, False), (F32, self.sz_shape, None, False)
        self._forward_form = _forms(*codes, column, (y_dtype, self.r_shape, self.r_strides, False), y, z, *zq, self.workspace_bytes)
        self._backward_form = _forms(y, *codes, z, *zq, (x_dtype, self.x_shape, self.x_strides, False),
                                     (x_dtype, self.w_shape, None, False), column, self.backward_workspace_bytes)

    def empty_input(self, device="cuda"):
        """A tensor of dx's form."""
        return _empty(self.x_shape, self.x_stride, self.x_dtype, device)

    def empty_output(self, device="cuda"):
        return _empty(self.y_shape, self.y_stride, self.y_dtype, device)

    def empty_z(self, device="cuda"):
        """The product before its activation, as it is."""
        return torch.empty(self.y_shape, dtype=self.y_dtype, device=device)

    def empty_z_codes(self, device="cuda"):
        """(zq, sz): the same in codes, a scale for every 32 columns."""
        return _empty_codes(self.zq_shape, self.sz_shape, device)

    def empty_weight_gradient(self, device="cuda"):
        return torch.empty(self.w_shape, dtype=self.x_dtype, device=device)


def _empty_codes(code_shape, scale_shape, device):
    return (torch.empty(code_shape, dtype=torch.int8, device=device),
            torch.empty(scale_shape, dtype=torch.float32, device=device))


def wq8_quant_pack(plan: QuantPlan, x, codes=None, scales=None, stream=None):
    """(codes, scales)."""
    if stream is None and _given(plan._pack, plan._h, plan._pack_form, x, codes, scales):
        return codes, scales
    a = _Args(stream)
    px = a.need(x, "x", plan.x_dtype, plan.x_shape, plan.x_strides)
    if codes is None:
        codes = a.make(torch.empty, plan.code_shape, dtype=torch.int8, device=x.device)
    if scales is None:
        scales = a.make(torch.empty, plan.scale_shape, dtype=torch.float32, device=x.device)
    pc = a.need(codes, "codes", torch.int8, plan.code_shape)
    ps = a.need(scales, "scales", torch.float32, plan.scale_shape)
    a.call(plan._pack, (plan._h, px, pc, ps))
    return codes, scales


def wq8_quant_unpack(plan: QuantPlan, codes, scales, x=None, stream=None):
    """x, the values that the codes stand for."""
    if stream is None and _given(plan._unpack, plan._h, plan._unpack_form, codes, scales, x):
        return x
    a = _Args(stream)
    pc = a.need(codes, "codes", torch.int8, plan.code_shape)
    ps = a.need(scales, "scales", torch.float32, plan.scale_shape)
    if x is None:
        x = a.make(plan.empty_input, codes.device)
    px = a.need(x, "x", plan.x_dtype, plan.x_shape, plan.x_strides)
    a.call(plan._unpack, (plan._h, pc, ps, px))
    return x


def wq8_rms_forward(plan: RmsPlan, x, gamma=None, residual=None, y=None, h=None, codes=None, scales=None, rstd=None,
                    want_y=True, want_codes=False, want_rstd=False, workspace=None, stream=None):
    """(y, h, codes, scales, rstd); what is neither given nor wanted is None. The
    stream h is made where a residual is given (it may be x or residual itself);
    without one it is x."""
    if (stream is None and not (want_y and y is None) and not (want_codes and codes is None) and not (want_rstd and rstd is None) and
            (h is None) == (residual is None) and (codes is None) == (scales is None) and
            _given(plan._forward, plan._h, plan._forward_form, x, residual, gamma, h, y, codes, scales, rstd, workspace)):
        return y, x if residual is None else h, codes, scales, rstd
    f32 = torch.float32
    a = _Args(stream)
    px = a.need(x, "x", plan.x_dtype, plan.x_shape, plan.x_strides)
    pr = a.optional(residual, "residual", plan.x_dtype, plan.x_shape, plan.x_strides)
    pg = a.optional(gamma, "gamma", f32, (plan.C,))
    if h is None and residual is not None:
        h = a.make(plan.empty_input, x.device)
    if y is None and want_y:
        y = a.make(plan.empty_output, x.device)
    if codes is None and want_codes:
        codes = a.make(torch.empty, plan.code_shape, dtype=torch.int8, device=x.device)
    if scales is None and codes is not None:
        scales = a.make(torch.empty, plan.scale_shape, dtype=f32, device=x.device)
    if rstd is None and want_rstd:
        rstd = a.make(torch.empty, plan.rows, dtype=f32, device=x.device)
    ph = a.optional(h, "h", plan.x_dtype, plan.x_shape, plan.x_strides)
    py = a.optional(y, "y", plan.y_dtype, plan.y_shape, plan.y_strides)
    pc = a.optional(codes, "codes", torch.int8, plan.code_shape)
    ps = a.optional(scales, "scales", f32, plan.scale_shape)
    pd = a.optional(rstd, "rstd", f32, (plan.rows,))
    ws, nw = a.workspace(workspace, plan.workspace_bytes)
    a.call(plan._forward, (plan._h, px, pr, pg, ph, py, pc, ps, pd, ws, nw))
    return y, x if residual is None else h, codes, scales, rstd


def wq8_rms_backward(plan: RmsPlan, dy, h, rstd, gamma=None, dh=None, dx=None, dgamma=None, workspace=None, stream=None):
    """(dx, dgamma). dx, which may be dh itself, is the gradient of x and of the
    residual; dgamma is made where gamma is given."""
    if stream is None and (dgamma is not None or gamma is None) and _given(
            plan._backward, plan._h, plan._backward_form, dy, h, rstd, gamma, dh, dx, dgamma, workspace):
        return dx, dgamma
    f32 = torch.float32
    a = _Args(stream)
    pdy = a.need(dy, "dy", plan.y_dtype, plan.y_shape, plan.y_strides)
    ph = a.need(h, "h", plan.x_dtype, plan.x_shape, plan.x_strides)
    pr = a.need(rstd, "rstd", f32, (plan.rows,))
    pg = a.optional(gamma, "gamma", f32, (plan.C,))
    pdh = a.optional(dh, "dh", plan.x_dtype, plan.x_shape, plan.x_strides)
    if dx is None:
        dx = a.make(plan.empty_input, h.device)
    if dgamma is None and gamma is not None:
        dgamma = a.make(torch.empty, plan.C, dtype=f32, device=h.device)
    pdx = a.need(dx, "dx", plan.x_dtype, plan.x_shape, plan.x_strides)
    pdg = a.optional(dgamma, "dgamma", f32, (plan.C,))
    ws, nw = a.workspace(workspace, plan.backward_workspace_bytes)
    a.call(plan._backward, (plan._h, pdy, ph, pr, pg, pdh, pdx, pdg, ws, nw))
    return dx, dgamma


def wq8_q8linear_forward(plan: Q8LinearPlan, xq, sx, wq, sw, bias=None, residual=None, y=None, z=None, zq=None, sz=None,
                         want_z=False, want_zq=False, workspace=None, stream=None):
    """y, with want_z (y, z), with want_zq (y, zq, sz), with both (y, z, zq, sz)."""
    if stream is None and not want_z and not want_zq and (zq is None) == (sz is None) and _given(
            plan._forward, plan._h, plan._forward_form, xq, sx, wq, sw, bias, residual, y, z, zq, sz, workspace):
        return y
    i8, f32 = torch.int8, torch.float32
    a = _Args(stream)
    px = a.need(xq, "xq", i8, plan.xq_shape)
    psx = a.need(sx, "sx", f32, (plan.rows,))
    pw = a.need(wq, "wq", i8, plan.wq_shape)
    psw = a.need(sw, "sw", f32, (plan.Cout,))
    pb = a.optional(bias, "bias", f32, (plan.Cout,))
    pr = a.optional(residual, "residual", plan.y_dtype, plan.r_shape, plan.r_strides)
    if y is None:
        y = a.make(plan.empty_output, xq.device)
    if z is None and want_z:
        z = a.make(plan.empty_z, xq.device)
    if zq is None and want_zq:
        zq = a.make(torch.empty, plan.zq_shape, dtype=i8, device=xq.device)
    if sz is None and zq is not None:
        sz = a.make(torch.empty, plan.sz_shape, dtype=f32, device=xq.device)
    py = a.need(y, "y", plan.y_dtype, plan.y_shape, plan.y_strides)
    pz = a.optional(z, "z", plan.y_dtype, plan.y_shape)
    pzq = a.optional(zq, "zq", i8, plan.zq_shape)
    psz = a.optional(sz, "sz", f32, plan.sz_shape)
    ws, nw = a.workspace(workspace, plan.workspace_bytes)
    a.call(plan._forward, (plan._h, px, psx, pw, psw, pb, pr, py, pz, pzq, psz, ws, nw))
    out = (y,) + ((z,) if want_z else ()) + ((zq, sz) if want_zq else ())
    return out if len(out) > 1 else y


def wq8_q8linear_backward(plan: Q8LinearPlan, dy, xq, sx, wq, sw, z=None, zq=None, sz=None, dx=None, dw=None, dbias=None,
                          want_dx=True, want_dw=True, want_dbias=False, workspace=None, stream=None):
    """(dx, dw, dbias); what is neither given nor wanted is None. z, or (zq, sz):
    what the forward kept, unless act is "none"."""
    none = plan.act == "none"
    if (stream is None and (none or (z is None) != (zq is None)) and (zq is None) == (sz is None) and
            not (want_dx and dx is None) and not (want_dw and dw is None) and not (want_dbias and dbias is None) and
            _given(plan._backward, plan._h, plan._backward_form, dy, xq, sx, wq, sw, None if none else z, None if none else zq,
                   None if none else sz, dx, dw, dbias, workspace)):
        return dx, dw, dbias
    i8, f32 = torch.int8, torch.float32
    a = _Args(stream)
    pdy = a.need(dy, "dy", plan.y_dtype, plan.y_shape, plan.y_strides)
    px = a.need(xq, "xq", i8, plan.xq_shape)
    psx = a.need(sx, "sx", f32, (plan.rows,))
    pw = a.need(wq, "wq", i8, plan.wq_shape)
    psw = a.need(sw, "sw", f32, (plan.Cout,))
    pz = pzq = psz = None
    if plan.act != "none":
        if zq is None:
            pz = a.need(z, "z", plan.y_dtype, plan.y_shape)
        else:
            if z is not None:
                raise ValueError("z and zq are given: one of the two")
            pzq = a.need(zq, "zq", i8, plan.zq_shape)
            psz = a.need(sz, "sz", f32, plan.sz_shape)
    if dx is None and want_dx:
        dx = a.make(plan.empty_input, xq.device)
    if dw is None and want_dw:
        dw = a.make(plan.empty_weight_gradient, xq.device)
    if dbias is None and want_dbias:
        dbias = a.make(torch.empty, plan.Cout, dtype=f32, device=xq.device)
    pdx = a.optional(dx, "dx", plan.x_dtype, plan.x_shape, plan.x_strides)
    pdw = a.optional(dw, "dw", plan.x_dtype, plan.w_shape)
    pdb = a.optional(dbias, "dbias", f32, (plan.Cout,))
    ws, nw = a.workspace(workspace, plan.backward_workspace_bytes)
    a.call(plan._backward, (plan._h, pdy, px, psx, pw, psw, pz, pzq, psz, pdx, pdw, pdb, ws, nw))
    return dx, dw, dbias
