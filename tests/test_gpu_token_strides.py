"""Tensors that are slices of wider ones, through every kernel of the operators on
8-bit codes: as contiguous ones to the bit, and nothing between the rows is written."""
import pytest
import token_plan_cases as P
import torch

import quantized_convolution_amd as q

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
WHOLE = [(1024, 256, 1024), (2048, 256, 4096), (256, 8192, 256), (64, 1024, 640)]  # whole tiles alone, and split


@pytest.fixture(scope="module", autouse=True)
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.load()


class Wide:
    """t in rows of `stride` elements; what lies between is 77."""

    def __init__(self, t, stride):
        self.base = torch.full((t.shape[0], stride), 77.0, dtype=t.dtype, device="cuda")
        self.t = self.base[:, :t.shape[1]]
        self.t.copy_(t)

    def untouched(self):
        return bool((self.base[:, self.t.shape[1]:] == 77).all())


def operands(rows, Cin, Cout, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + Cin + Cout)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, w = r(rows, Cin), r(Cout, Cin) / Cin ** 0.5
    a = q.wq8_quant_pack(q.QuantPlan(rows, Cin), x) + q.wq8_quant_pack(q.QuantPlan(Cout, Cin), w)
    return a, r(Cout), r(rows, Cout).to(dtype), r(rows, Cout).to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows,Cin,Cout", P.FORWARD + WHOLE)
def test_forward(rows, Cin, Cout, dtype):
    print("[case] strides", rows, Cin, Cout, dtype, flush=True)
    a, bias, residual, _ = operands(rows, Cin, Cout, dtype)
    act = "silu" if rows % 2 else "none"
    want = q.wq8_q8linear_forward(q.Q8LinearPlan(rows, Cin, Cout, act, x_dtype=dtype), *a, bias, residual, want_z=True, want_zq=True)
    for ys, rs in ((0, Cout + 5), (Cout + 3, 0), (Cout + 8, Cout + 16), (Cout + 1, Cout + 2)):
        p = q.Q8LinearPlan(rows, Cin, Cout, act, x_dtype=dtype, y_stride=ys, r_stride=rs)
        r, y = Wide(residual, rs or Cout), Wide(torch.zeros_like(residual), ys or Cout)
        z, (zq, sz) = p.empty_z(), p.empty_z_codes()
        zq.fill_(55)
        q.wq8_q8linear_forward(p, *a, bias, r.t, y=y.t, z=z, zq=zq, sz=sz)
        for got, w, what in zip((y.t, z, zq, sz), want, ("y", "z", "zq", "sz")):
            assert torch.equal(got, w), (what, ys, rs)
        assert y.untouched() and r.untouched() and torch.equal(r.t, residual)
        y.t.fill_(0)
        assert torch.equal(q.wq8_q8linear_forward(p, *a, bias, r.t, y=y.t), want[0])
    for s in (Cout + 7, Cout + 8):  # the residual is y
        p = q.Q8LinearPlan(rows, Cin, Cout, act, x_dtype=dtype, y_stride=s, r_stride=s)
        over = Wide(residual, s)
        q.wq8_q8linear_forward(p, *a, bias, over.t, y=over.t)
        assert torch.equal(over.t, want[0]) and over.untouched()
    if rows % 2 == 0:  # a planar residual in front of rows that are apart
        pixels = rows // 2
        p = q.Q8LinearPlan(rows, Cin, Cout, act, x_dtype=dtype, r_layout="nchw", pixels=pixels, y_stride=Cout + 3)
        y = Wide(torch.zeros_like(residual), Cout + 3)
        planar = residual.view(2, pixels, Cout).permute(0, 2, 1).contiguous()
        q.wq8_q8linear_forward(p, *a, bias, planar, y=y.t)
        assert torch.equal(y.t, want[0]) and y.untouched()


def backward(dtype, rows, Cin, Cout, round_dz):
    print("[case] strides backward", dtype, rows, Cin, Cout, round_dz, flush=True)
    a, _, dy, z = operands(rows, Cin, Cout, dtype)
    make = lambda **kw: q.Q8LinearPlan(rows, Cin, Cout, "relu", x_dtype=dtype, round_dz=round_dz, **kw)  # noqa: E731
    want = q.wq8_q8linear_backward(make(), dy, *a, z=z, want_dbias=True)
    for xs, ys in ((Cin + 5, 0), (0, Cout + 3), (Cin + 8, Cout + 8)):
        p = make(x_stride=xs, y_stride=ys)
        d, dx = Wide(dy, ys or Cout), Wide(torch.zeros(rows, Cin, dtype=dtype, device="cuda"), xs or Cin)
        _, dw, db = q.wq8_q8linear_backward(p, d.t, *a, z=z, dx=dx.t, want_dbias=True)
        assert torch.equal(dx.t, want[0]) and torch.equal(dw, want[1]) and torch.equal(db, want[2])
        assert dx.untouched() and d.untouched()


@pytest.mark.parametrize("dtype,rows,Cin,Cout", [(DT, *c) for DT, t in ((F32, "f32"), (BF, "bf16")) for c in P.BACKWARD[t] + WHOLE])
def test_backward(dtype, rows, Cin, Cout):
    backward(dtype, rows, Cin, Cout, False)


@pytest.mark.parametrize("rows,Cin,Cout", P.BACKWARD["bf16"] + WHOLE)
def test_backward_of_rounded_dz(rows, Cin, Cout):
    backward(BF, rows, Cin, Cout, True)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("C", P.ROWS + [8, 2048, 8192])
def test_rows(C, dtype):
    """The norm and its backward, packing and unpacking."""
    print("[case] strided rows", C, dtype, flush=True)
    g = torch.Generator(device="cuda").manual_seed(C)
    x, res, dy = (torch.randn(9, C, generator=g, device="cuda").to(dtype) for _ in range(3))
    gm = 1 + 0.2 * torch.randn(C, generator=g, device="cuda")
    plain = q.RmsPlan(9, C, x_dtype=dtype)
    want = q.wq8_rms_forward(plain, x, gm, res, want_codes=True, want_rstd=True)
    grads = q.wq8_rms_backward(plain, dy, want[1], want[4], gm, dh=res)
    for xs, ys in ((C + 3, C + 8), (C + 8, C + 1)):
        p = q.RmsPlan(9, C, x_dtype=dtype, x_stride=xs, y_stride=ys)
        wx, wr, wh, wy, wd, wdx = (Wide(t, s) for t, s in ((x, xs), (res, xs), (x, xs), (x, ys), (dy, ys), (x, xs)))
        got = q.wq8_rms_forward(p, wx.t, gm, wr.t, y=wy.t, h=wh.t, want_codes=True, want_rstd=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        dx, dg = q.wq8_rms_backward(p, wd.t, wh.t, got[4], gm, dh=wr.t, dx=wdx.t)
        assert torch.equal(dx, grads[0]) and torch.equal(dg, grads[1])
        assert all(w.untouched() for w in (wx, wr, wh, wy, wd, wdx))
    for group in (0, 32, 64, 128):
        codes = q.wq8_quant_pack(q.QuantPlan(9, C, group, x_dtype=dtype), x)
        values = q.wq8_quant_unpack(q.QuantPlan(9, C, group, x_dtype=dtype), *codes)
        p, wx, out = q.QuantPlan(9, C, group, x_dtype=dtype, x_stride=C + 5), Wide(x, C + 5), Wide(x, C + 5)
        got = q.wq8_quant_pack(p, wx.t)
        assert torch.equal(got[0], codes[0]) and torch.equal(got[1], codes[1])
        assert torch.equal(q.wq8_quant_unpack(p, *got, x=out.t), values) and out.untouched() and wx.untouched()
