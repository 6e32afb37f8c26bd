"""Every kernel instance of the operators on 8-bit codes that a plan can choose
(token_plan_cases.py, held to that by test_token_plan_cases.py), against 64 bits.
The reference runs on the GPU, in plain products of two matrices."""
import pytest
import token_plan_cases as P
import token_reference as R
import torch

import quantized_convolution_amd as q

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
DT = {"f32": F32, "bf16": BF}


@pytest.fixture(scope="module", autouse=True)
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.load()


def check(got, pair, what):
    want, bound = pair
    bad = ~((got.double() - want).abs() <= bound)
    assert got.shape == want.shape and not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()}"


def operands(seed, rows, Cin, Cout):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, w = r(rows, Cin) * (1 + 15 * (torch.rand(rows, Cin, generator=g, device="cuda") < 0.01)), r(Cout, Cin) / Cin ** 0.5
    return q.wq8_quant_pack(q.QuantPlan(rows, Cin), x), q.wq8_quant_pack(q.QuantPlan(Cout, Cin), w), r


def product(xq, sx, wq, sw, Cin, bias):
    acc = xq[:, :Cin].double() @ wq[:, :Cin].double().T
    return acc.float() * sx[:, None] * sw[None, :] + bias


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,Cin,Cout", P.FORWARD)
def test_forward(rows, Cin, Cout, dtype):
    print("[case] product", rows, Cin, Cout, dtype, flush=True)
    (xq, sx), (wq, sw), r = operands(rows + Cin, rows, Cin, Cout)
    bias, residual = r(Cout), r(rows, Cout).to(DT[dtype])
    for act in ("gelu", "none"):
        p = q.Q8LinearPlan(rows, Cin, Cout, act, x_dtype=DT[dtype])
        zq, sz = p.empty_z_codes()
        zq.fill_(55)
        y, z, zq, sz = q.wq8_q8linear_forward(p, xq, sx, wq, sw, bias, residual, zq=zq, sz=sz, want_z=True, want_zq=True)
        want = product(xq, sx, wq, sw, Cin, bias)
        assert torch.equal(z, want.to(DT[dtype]))
        assert zq.shape == p.zq_shape
        codes, scales = q.wq8_quant_pack(q.QuantPlan(rows, Cout, group=32), want)
        assert torch.equal(zq, codes) and torch.equal(sz, scales)
        check(y, R.forward(want, act, residual, DT[dtype]), "y")
        over = residual.clone()
        q.wq8_q8linear_forward(p, xq, sx, wq, sw, bias, over, y=over)
        assert torch.equal(over, y)


@pytest.mark.parametrize("kept", ["codes", "values"])
@pytest.mark.parametrize("dtype,rows,Cin,Cout", [(t, *c) for t, cases in P.BACKWARD.items() for c in cases])
def test_backward(dtype, rows, Cin, Cout, kept):
    print("[case] product backward", dtype, rows, Cin, Cout, kept, flush=True)
    (xq, sx), (wq, sw), r = operands(rows + Cout, rows, Cin, Cout)
    z, dy = product(xq, sx, wq, sw, Cin, 0.0), r(rows, Cout).to(DT[dtype])
    dy[rows // 2] = 0
    p = q.Q8LinearPlan(rows, Cin, Cout, "gelu", x_dtype=DT[dtype])
    if kept == "codes":
        zq, sz = q.wq8_quant_pack(q.QuantPlan(rows, Cout, group=32), z)
        kw, zz = dict(zq=zq, sz=sz), zq[:, :Cout].float() * sz.repeat_interleave(32, 1)[:, :Cout]
    else:
        zz = z.to(DT[dtype])
        kw = dict(z=zz)
    ws = p.empty_backward_workspace()
    ws.fill_(0x5A)
    dx, dw, db = q.wq8_q8linear_backward(p, dy, xq, sx, wq, sw, **kw, want_dbias=True, workspace=ws)
    want = R.backward(dy, xq, sx, wq, sw, Cin, DT[dtype], "gelu", zz)
    check(dx, want["dx"], "dx")
    check(dw, want["dw"], "dw")
    check(db, want["dbias"], "dbias")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", P.ROWS)
def test_rows(C, dtype):
    """Whole and odd widths around each shape's, more rows than a block has."""
    print("[case] rows", C, dtype, flush=True)
    g = torch.Generator().manual_seed(C)
    for width in (C, C + 1, C - C % 8 or 8):
        x, res, dy = (torch.randn(9, width, generator=g).to(DT[dtype]) for _ in range(3))
        gm = 1 + 0.2 * torch.randn(width, generator=g)
        h = (x.float() + res.float()).to(DT[dtype])
        p = q.RmsPlan(9, width, x_dtype=DT[dtype])
        y, got, codes, scales, rstd = q.wq8_rms_forward(p, x.cuda(), gm.cuda(), res.cuda(), want_codes=True, want_rstd=True)
        ref = R.Rms(h, 1e-6, gm)
        assert torch.equal(got.cpu(), h)
        check(rstd.cpu(), ref.forward(DT[dtype])["rstd"], "rstd")
        check(y.cpu(), ref.forward(DT[dtype])["y"], "y")
        t = R.codes_of(h.float().numpy() * gm.numpy())
        assert torch.equal(codes.cpu(), t[0])
        check(scales.cpu(), ref.scales(t[1]), "scales")
        dx, dg = q.wq8_rms_backward(p, dy.cuda(), got, rstd, gm.cuda(), dh=res.cuda())
        want = ref.backward(dy, rstd.cpu(), res, DT[dtype])
        check(dx.cpu(), want["dx"], "dx")
        check(dg.cpu(), want["dgamma"], "dgamma")
        plain = q.wq8_quant_pack(q.QuantPlan(9, width, x_dtype=DT[dtype]), x.cuda())
        t = R.codes_of(x.float().numpy())
        assert torch.equal(plain[0].cpu(), t[0]) and torch.equal(plain[1].cpu(), t[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [333, 1290, 2100, 5000, 9000, 15001])
def test_backward_rows_in_turn(C, dtype):
    """Several rows a wave or block, one after the other, the last block with fewer."""
    print("[case] rows in turn", C, dtype, flush=True)
    rows = 4801 if C < 2048 else 601
    g = torch.Generator().manual_seed(C)
    h, dh, dy = (torch.randn(rows, C, generator=g).to(DT[dtype]) for _ in range(3))
    gm = 1 + 0.2 * torch.randn(C, generator=g)
    p = q.RmsPlan(rows, C, x_dtype=DT[dtype])
    rstd = q.wq8_rms_forward(p, h.cuda(), gm.cuda(), want_rstd=True)[4]
    dx, dg = q.wq8_rms_backward(p, dy.cuda(), h.cuda(), rstd, gm.cuda(), dh=dh.cuda())
    want = R.Rms(h, 1e-6, gm).backward(dy, rstd.cpu(), dh, DT[dtype])
    check(dx.cpu(), want["dx"], "dx")
    check(dg.cpu(), want["dgamma"], "dgamma")
