"""The operators on 8-bit codes on the GPU: codes to the bit, everything else
against 64 bits within bounds of fp32 rounding (token_reference.py)."""
import numpy as np
import pytest
import torch
import token_reference as R

import quantized_convolution_amd as q

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
DT = {"f32": F32, "bf16": BF}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.load()
    return torch.device("cuda:0")


def say(*a):
    print("[case]", *a, flush=True)


def rand(g, *shape):
    """Normal values, a few of them far out."""
    v = torch.randn(shape, generator=g)
    return v * (1 + 15 * (torch.rand(shape, generator=g) < 0.01))


def wide(t, stride, dev):
    """t on the GPU in rows of `stride` elements; what lies between is 77."""
    if not stride:
        return t.to(dev).contiguous()
    w = torch.full((t.shape[0], stride), 77.0, dtype=t.dtype, device=dev)
    w[:, :t.shape[1]] = t.to(dev)
    return w[:, :t.shape[1]]


def untouched(t, stride):
    """Whether what lies between the rows of wide()'s tensor is as it was."""
    if not stride or t.shape[0] < 2:
        return True
    base = t.as_strided((t.shape[0] - 1, stride), (stride, 1))
    return bool((base[:, t.shape[1]:] == 77).all())


def check(got, want, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{what}{at}: {got[at].item()!r} for {want[at].item()!r}, bound "
                             f"{(bound[at] if isinstance(bound, torch.Tensor) else bound)!r}; {int(bad.sum())} of {bad.numel()}")


def same(got, want, what):
    got = got.detach().cpu()
    eq = (got == want) | (torch.isnan(got.float()) & torch.isnan(want.float()))
    assert got.shape == want.shape and bool(eq.all()), f"{what}: {int((~eq).sum())} of {eq.numel()} differ"


# ---------------------------------------------------------------------- pack
PACK = [(1, 1, 0), (3, 7, 0), (5, 8, 0), (4, 9, 32), (7, 31, 32), (7, 33, 32), (6, 64, 64), (9, 130, 64), (5, 127, 128),
        (3, 129, 128), (2, 300, 128), (77, 333, 0), (65, 511, 0), (9, 513, 0), (33, 1024, 0), (5, 2047, 0), (3, 2565, 32),
        (2, 4096, 0), (2, 4097, 0), (3, 8191, 0), (2, 10240, 0), (2, 16385, 0), (1, 33000, 0), (1001, 40, 32), (3, 6, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C,group", PACK)
def test_pack_and_unpack(dev, rows, C, group, dtype):
    say("pack", rows, C, group, dtype)
    g = torch.Generator().manual_seed(rows * 1000 + C)
    extra = C + 5 if (rows + C) % 2 else 0
    x = rand(g, rows, C).to(DT[dtype])
    x[0, : max(1, C // 2)] = 0  # whole groups of zeros
    plan = q.QuantPlan(rows, C, group=group, x_dtype=DT[dtype], x_stride=extra)
    codes, scales = plan.empty_codes(dev)
    codes.fill_(55)
    q.wq8_quant_pack(plan, wide(x, extra, dev), codes=codes, scales=scales)
    wc, ws = R.codes_of(x.float().numpy(), group)
    same(codes, wc, "codes")
    same(scales, ws, "scales")
    out = wide(torch.zeros(rows, C, dtype=DT[dtype]), extra, dev)
    q.wq8_quant_unpack(plan, codes, scales, x=out)
    want = wc[:, :C].float() * (ws.repeat_interleave(group, 1)[:, :C] if group else ws[:, None])
    same(out, want.to(DT[dtype]), "x")
    assert untouched(out, extra)
    a = plan.empty_input(dev)
    made = q.wq8_quant_pack(plan, wide(x, extra, dev))
    same(made[0], wc, "codes made here")
    same(q.wq8_quant_unpack(plan, *made), want.to(DT[dtype]), "x made here")
    assert a.shape == out.shape and a.stride() == out.stride()


@pytest.mark.parametrize("group", [0, 32])
def test_pack_borders(dev, group):
    """Ties, denormals, the largest and smallest numbers, infinities and NaN."""
    say("pack borders", group)
    C = 96
    x = torch.zeros(10, C)
    x[0, :40] = torch.arange(40) + 0.5
    x[0, 95] = 127.0
    x[0, 64] = -127.0
    x[1] = torch.linspace(-3e38, 3e38, C)
    x[2] = torch.arange(C).float() * 2.0 ** -149
    x[3, 5] = 2.0 ** -149
    x[4] = torch.linspace(-1, 1, C) * 2.0 ** -122
    x[5] = torch.linspace(-1, 1, C) * 2.0 ** -100
    x[6] = 1.0
    x[6, 40] = float("inf")
    x[7] = 1.0
    x[7, 41] = float("nan")
    x[8] = float("-inf")
    x[9] = -0.0
    plan = q.QuantPlan(10, C, group=group)
    codes, scales = q.wq8_quant_pack(plan, x.to(dev))
    wc, ws = R.codes_of(x.numpy(), group)
    same(codes, wc, "codes")
    same(scales, ws, "scales")
    back = q.wq8_quant_unpack(plan, codes, scales).cpu()
    for r in (6, 7, 8):
        lo, hi = (32, 64) if group and r < 8 else (0, C)
        assert torch.isnan(back[r, lo:hi]).all()
    if group:
        assert torch.isfinite(back[6, :32]).all() and torch.isfinite(back[7, 64:]).all()


# ---------------------------------------------------------------------- norm
NORM = [(1, 1), (5, 7), (3, 8), (1, 1280), (6, 9), (77, 333), (130, 512), (9, 640), (65, 1001), (4, 1285), (33, 2048), (5, 2560),
        (3, 4095), (2, 5120), (2, 8193), (3, 10240), (2, 16392), (1, 33001)]


@pytest.mark.parametrize("types", ["f32/f32", "bf16/bf16", "bf16/f32", "f32/bf16"])
@pytest.mark.parametrize("rows,C", NORM)
def test_norm_forward(dev, rows, C, types):
    say("norm", rows, C, types)
    xt, yt = (DT[t] for t in types.split("/"))
    g = torch.Generator().manual_seed(rows * 7 + C)
    for residual, gamma, xs, ys in ((False, True, 0, 0), (True, True, C + 3, 0), (True, False, 0, C + 8)):
        x, r = rand(g, rows, C).to(xt), rand(g, rows, C).to(xt)
        gm = 1 + 0.2 * torch.randn(C, generator=g) if gamma else None
        h = (x.float() + r.float()).to(xt) if residual else x
        p = q.RmsPlan(rows, C, 1e-6, xt, yt, x_stride=xs, y_stride=ys)
        codes, scales = p.empty_codes(dev)
        codes.fill_(55)
        y, hout = wide(torch.zeros(rows, C, dtype=yt), ys, dev), wide(torch.zeros(rows, C, dtype=xt), xs, dev)
        got = q.wq8_rms_forward(p, wide(x, xs, dev), None if gm is None else gm.to(dev), wide(r, xs, dev) if residual else None,
                                y=y, h=hout if residual else None, codes=codes, scales=scales, want_rstd=True)
        ref = R.Rms(h, 1e-6, gm)
        if residual:
            same(hout, h, "h")
            assert untouched(hout, xs)
        f = ref.forward(yt)
        check(got[4], *f["rstd"], "rstd")
        check(y, *f["y"], "y")
        assert untouched(y, ys)
        t = h.float().numpy() * (gm.numpy()[None, :] if gamma else np.float32(1))
        wc, ws = R.codes_of(t)
        same(codes, wc, "codes")
        check(scales, *ref.scales(ws), "scales")
        # each output alone gives the same
        alone = q.wq8_rms_forward(p, wide(x, xs, dev), None if gm is None else gm.to(dev), wide(r, xs, dev) if residual else None,
                                  want_y=False, want_codes=True)
        assert alone[0] is None and alone[4] is None
        same(alone[2], wc, "codes alone")
        same(alone[3], scales.cpu(), "scales alone")
        same(q.wq8_rms_forward(p, wide(x, xs, dev), None if gm is None else gm.to(dev), wide(r, xs, dev) if residual else None)[0],
             y.cpu(), "y alone")


@pytest.mark.parametrize("C", [9, 520, 1285, 5121, 33001])
@pytest.mark.parametrize("which", ["x", "residual"])
def test_norm_in_place(dev, C, which):
    """The stream over x or over the residual."""
    say("norm in place", C, which)
    g = torch.Generator().manual_seed(C)
    x, r = rand(g, 5, C).to(BF), rand(g, 5, C).to(BF)
    p = q.RmsPlan(5, C, x_dtype=BF)
    gx, gr = x.to(dev), r.to(dev)
    y, h, codes, scales, _ = q.wq8_rms_forward(p, gx, None, gr, h=gx if which == "x" else gr, want_codes=True)
    want = q.wq8_rms_forward(p, x.to(dev), None, r.to(dev), want_codes=True)
    assert h is (gx if which == "x" else gr)
    for a, b in zip((y, h, codes, scales), want):
        same(a, b.cpu(), "in place")


def test_norm_borders(dev):
    """Rows of zeros, of tiny and of huge values, infinities and NaN: as the formulas give them, row by row."""
    say("norm borders")
    C = 200
    x = torch.ones(8, C)
    x[0] = 0
    x[1] = 1e-30
    x[2] = 3e38
    x[3, 7] = float("inf")
    x[4, 7] = float("nan")
    x[5] = 1e18
    x[6] = torch.linspace(-1, 1, C)
    gm = torch.ones(C)
    for eps in (1e-6, 0.0):
        p = q.RmsPlan(8, C, eps)
        y, h, codes, scales, rstd = (t.cpu() for t in q.wq8_rms_forward(p, x.to(dev), gm.to(dev), want_codes=True, want_rstd=True))
        with np.errstate(all="ignore"):
            r32 = 1 / torch.sqrt((x * x).sum(1) / C + eps)
            want = x * r32[:, None]
        assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(torch.isinf(rstd), torch.isinf(r32))
        ok = torch.isfinite(want).all(1)
        check(y[ok], want[ok].double(), (R.RSTD + 8) * R.U * want[ok].double().abs() + 1e-44, "y")
        wc, ws = R.codes_of(x.numpy())
        same(codes, wc, "codes")
        assert torch.equal(torch.isnan(scales), torch.isnan(ws * r32)) and torch.isnan(scales[3:5]).all()
        # what the codes stand for is y to half a code
        for i in (1, 5, 6) if eps else (5, 6):
            v = R.values(codes, scales, C)[i]
            assert bool(((v - y[i].double()).abs() <= scales[i].double() * 0.5 * (1 + 1e-4) + 1e-40).all())


BWD = [(1, 1), (3, 7), (5, 8), (1, 1280), (77, 333), (130, 512), (9, 640), (700, 100), (65, 1001), (5, 2048), (6, 2565), (3, 4097),
       (2, 8191), (3, 10240), (5, 33001), (4000, 64), (3100, 16)]


@pytest.mark.parametrize("types", ["f32/f32", "bf16/bf16", "bf16/f32", "f32/bf16"])
@pytest.mark.parametrize("rows,C", BWD)
def test_norm_backward(dev, rows, C, types):
    say("norm backward", rows, C, types)
    xt, yt = (DT[t] for t in types.split("/"))
    g = torch.Generator().manual_seed(rows * 3 + C)
    for gamma, with_dh, xs, ys in ((True, True, 0, C + 5), (True, False, C + 1, 0), (False, True, 0, 0)):
        h, dy, dh = rand(g, rows, C).to(xt), rand(g, rows, C).to(yt), rand(g, rows, C).to(xt)
        dy[rows // 2] = 0  # a row without a gradient
        gm = 1 + 0.2 * torch.randn(C, generator=g) if gamma else None
        ref = R.Rms(h, 1e-6, gm)
        rstd = ref.rstd.float()
        p = q.RmsPlan(rows, C, 1e-6, xt, yt, x_stride=xs, y_stride=ys)
        dx = wide(torch.zeros(rows, C, dtype=xt), xs, dev)
        dg = torch.full((C,), 9.0, device=dev)
        a = (p, wide(dy, ys, dev), wide(h, xs, dev), rstd.to(dev), None if gm is None else gm.to(dev))
        kw = dict(dh=wide(dh, xs, dev) if with_dh else None)
        q.wq8_rms_backward(*a, **kw, dx=dx, dgamma=dg)
        want = ref.backward(dy, rstd, dh if with_dh else None, xt)
        check(dx, *want["dx"], "dx")
        check(dg, *want["dgamma"], "dgamma")
        assert untouched(dx, xs)
        again = q.wq8_rms_backward(*a, **kw)
        same(again[0], dx.cpu(), "dx again")
        assert (again[1] is None) == (gm is None)
        if gm is not None:
            same(again[1], dg.cpu(), "dgamma again")
        if with_dh:  # over dh itself
            over = wide(dh, xs, dev)
            q.wq8_rms_backward(*a, dh=over, dx=over)
            same(over, dx.cpu(), "dx over dh")


def test_norm_gradient_is_the_slope(dev):
    """Against differences of the forward pass, in the direction of a random vector."""
    say("norm differences")
    rows, C = 7, 300
    g = torch.Generator().manual_seed(1)
    h, d, gm, dy = (torch.randn(s, generator=g) for s in ((rows, C), (rows, C), (C,), (rows, C)))
    p = q.RmsPlan(rows, C, 1e-6)
    rstd = q.wq8_rms_forward(p, h.to(dev), gm.to(dev), want_rstd=True)[4]
    dx, dg = q.wq8_rms_backward(p, dy.to(dev), h.to(dev), rstd, gm.to(dev))
    # the step's own error is eps^2 times a third derivative of order one, the difference's 2^-22 / eps of the sum
    eps = 2.0 ** -6
    for v, grad, at in ((d, dx, 0), (torch.randn(C, generator=g), dg, 1)):
        f = lambda s: (q.wq8_rms_forward(p, (h + (s * v if at == 0 else 0)).to(dev), (gm + (s * v if at else 0)).to(dev))[0].cpu().double()  # noqa: E731
                       * dy.double()).sum()
        diff = (f(eps) - f(-eps)) / (2 * eps)
        dot = (grad.cpu().double() * v.double()).sum()
        size = (grad.cpu().double() * v.double()).abs().sum()
        assert abs(diff - dot) <= 3 * eps ** 2 * size, (diff, dot)


# ------------------------------------------------------------------- product
# rows, Cin, Cout, act, residual, y_dtype
FWD = [
    (1, 1, 1, "none", "none", "f32"), (1, 640, 1280, "silu", "rows", "bf16"), (1, 5000, 77, "gelu", "planar", "f32"),
    (2, 127, 33, "none", "rows", "f32"), (16, 128, 31, "relu", "none", "bf16"), (17, 129, 64, "gelu_tanh", "rows", "bf16"),
    (33, 1285, 100, "silu", "planar", "f32"), (64, 2565, 321, "gelu", "rows", "bf16"), (77, 1285, 130, "gelu_tanh", "none", "f32"),
    (65, 64, 7, "none", "rows", "bf16"), (100, 40, 65, "none", "planar", "f32"), (130, 333, 515, "silu", "rows", "f32"),
    (200, 9000, 60, "none", "none", "bf16"), (1024, 256, 1001, "gelu", "rows", "bf16"), (300, 70000, 3, "none", "none", "f32"),
    (5, 70000, 40, "none", "none", "f32"), (2500, 384, 1300, "relu", "planar", "bf16"),
]


def make(g, rows, Cin, Cout):
    xq, sx = R.codes_of(rand(g, rows, Cin).numpy())
    wq, sw = R.codes_of(torch.randn(Cout, Cin, generator=g).numpy() / np.float32(np.sqrt(Cin)))
    return xq, sx, wq, sw


@pytest.mark.parametrize("rows,Cin,Cout,act,residual,y_dtype", FWD)
def test_product(dev, rows, Cin, Cout, act, residual, y_dtype):
    say("product", rows, Cin, Cout, act, residual, y_dtype)
    yt = DT[y_dtype]
    g = torch.Generator().manual_seed(rows + Cin + Cout)
    xq, sx, wq, sw = make(g, rows, Cin, Cout)
    bias = torch.randn(Cout, generator=g) if Cout % 2 else None
    pixels = max(d for d in (1, 2, 3, 5, 11, 25) if rows % d == 0) if residual == "planar" else 0
    ys = Cout + 3 if Cin % 2 else 0
    p = q.Q8LinearPlan(rows, Cin, Cout, act, x_dtype=yt, r_layout="nchw" if pixels else "nhwc", pixels=pixels, y_stride=ys)
    z = R.product(xq, sx, wq, sw, Cin, bias)
    r = rr = None
    if residual == "rows":
        r = rr = torch.randn(rows, Cout, generator=g).to(yt)
    elif pixels:
        r = torch.randn(rows // pixels, Cout, pixels, generator=g).to(yt)
        rr = r.permute(0, 2, 1).reshape(rows, Cout)
    y = wide(torch.zeros(rows, Cout, dtype=yt), ys, dev)
    zq, sz = p.empty_z_codes(dev)
    zq.fill_(55)
    zb = p.empty_z(dev)
    ws = torch.full((p.workspace_bytes,), 0x5A, dtype=torch.uint8, device=dev)
    args = [t.to(dev) for t in (xq, sx, wq, sw)] + [None if t is None else t.to(dev) for t in (bias, r)]
    q.wq8_q8linear_forward(p, *args, y=y, z=zb, zq=zq, sz=sz, workspace=ws)
    same(zb, z.to(yt), "z")
    wc, wsz = R.codes_of(z.numpy(), 32)
    same(zq, wc, "zq")
    same(sz, wsz, "sz")
    check(y, *R.forward(z, act, rr, yt), "y")
    assert untouched(y, ys)
    same(q.wq8_q8linear_forward(p, *args), y.cpu(), "y alone")
    got = q.wq8_q8linear_forward(p, *args, want_zq=True)
    same(got[1], wc, "zq made here")
    same(q.wq8_q8linear_forward(p, *args, want_z=True)[1], z.to(yt), "z made here")
    if residual == "rows":
        over = wide(r, ys, dev)
        if not ys:
            q.wq8_q8linear_forward(p, *args[:5], over, y=over)
            same(over, y.cpu(), "y over the residual")


def test_product_of_extreme_codes(dev):
    """Sums that pass 2^24, and nearly 2^31, are exact before they are rounded once."""
    say("extreme codes")
    for rows, Cin, Cout in ((3, 65536, 40), (3, 65664, 40), (100, 131072, 33), (100, 65536, 65)):
        xq = torch.full((rows, Cin), 127, dtype=torch.int8)
        wq = torch.full((Cout, Cin), 127, dtype=torch.int8)
        wq[1] = -127
        wq[2, ::2] = -126
        xq[1, 1::3] = 1
        sx, sw = torch.ones(rows), torch.ones(Cout)
        p = q.Q8LinearPlan(rows, Cin, Cout)
        y = q.wq8_q8linear_forward(p, *(t.to(dev) for t in (xq, sx, wq, sw)))
        same(y, (xq.double() @ wq.double().T).float(), "y")


def test_product_borders(dev):
    """A row that stands for NaN gives NaN there and nowhere else, a row of zeros the bias; in z's codes too."""
    say("product borders")
    for rows in (4, 100):
        g = torch.Generator().manual_seed(rows)
        x = torch.randn(rows, 200, generator=g)
        x[1, 3], x[2] = float("inf"), 0.0
        xq, sx = R.codes_of(x.numpy())
        wq, sw = R.codes_of(torch.randn(50, 200, generator=g).numpy())
        bias = torch.randn(50, generator=g)
        p = q.Q8LinearPlan(rows, 200, 50, "gelu")
        y, z, zq, sz = (t.cpu() for t in q.wq8_q8linear_forward(p, *(t.to(dev) for t in (xq, sx, wq, sw, bias)), want_z=True, want_zq=True))
        nan = torch.zeros(rows, 50, dtype=torch.bool)
        nan[1] = True
        assert torch.equal(torch.isnan(y), nan) and torch.equal(torch.isnan(z), nan)
        assert torch.equal(z[2], bias) and torch.isnan(sz[1]).all() and (zq[1] == 0).all()
        same(zq, R.codes_of(z.numpy(), 32)[0], "zq")


BWP = [
    (1, 1, 1, "none"), (1, 640, 1280, "silu"), (3, 127, 33, "gelu"), (77, 333, 130, "gelu_tanh"), (128, 128, 128, "none"),
    (129, 129, 65, "relu"), (200, 60, 7, "silu"), (1001, 333, 515, "silu"), (64, 2565, 321, "gelu"), (5000, 40, 24, "gelu"),
    (30, 8, 3000, "none"), (70000, 9, 5, "none"), (2048, 257, 1025, "gelu"),
]


@pytest.mark.parametrize("types", ["f32/f32", "bf16/bf16", "bf16/f32", "f32/bf16"])
@pytest.mark.parametrize("rows,Cin,Cout,act", BWP)
def test_product_backward(dev, rows, Cin, Cout, act, types):
    say("product backward", rows, Cin, Cout, act, types)
    xt, yt = (DT[t] for t in types.split("/"))
    g = torch.Generator().manual_seed(rows + 2 * Cin + Cout)
    xq, sx, wq, sw = make(g, rows, Cin, Cout)
    dy = rand(g, rows, Cout).to(yt)
    dy[rows // 2] *= 0.0 if rows > 2 else 1.0  # a row without a gradient
    dy[-1] *= 100.0
    ys, xs = (Cout + 3, Cin + 2) if rows % 2 else (0, 0)
    p = q.Q8LinearPlan(rows, Cin, Cout, act, x_dtype=xt, y_dtype=yt, x_stride=xs, y_stride=ys)
    z = R.product(xq, sx, wq, sw, Cin)
    for kept in ("codes", "values") if act != "none" else ("nothing",):
        kw, zz = {}, None
        if kept == "codes":
            zq, sz = R.codes_of(z.numpy(), 32)
            kw = dict(zq=zq.to(dev), sz=sz.to(dev))
            zz = zq[:, :Cout].float() * sz.repeat_interleave(32, 1)[:, :Cout]
        elif kept == "values":
            zz = z.to(yt)
            kw = dict(z=zz.to(dev))
        dx = wide(torch.zeros(rows, Cin, dtype=xt), xs, dev)
        dw = torch.full((Cout, Cin), 9.0, dtype=xt, device=dev)
        db = torch.full((Cout,), 9.0, device=dev)
        ws = torch.full((p.backward_workspace_bytes,), 0x5A, dtype=torch.uint8, device=dev)
        a = (p, wide(dy, ys, dev)) + tuple(t.to(dev) for t in (xq, sx, wq, sw))
        q.wq8_q8linear_backward(*a, **kw, dx=dx, dw=dw, dbias=db, workspace=ws)
        want = R.backward(dy, xq, sx, wq, sw, Cin, xt, act, zz)
        check(dx, *want["dx"], f"dx ({kept})")
        check(dw, *want["dw"], f"dw ({kept})")
        check(db, *want["dbias"], f"dbias ({kept})")
        assert untouched(dx, xs)
        # each alone gives the same, and again
        same(q.wq8_q8linear_backward(*a, **kw, want_dw=False)[0], dx.cpu(), "dx alone")
        one = q.wq8_q8linear_backward(*a, **kw, want_dx=False)
        assert one[0] is None and one[2] is None
        same(one[1], dw.cpu(), "dw alone")
        same(q.wq8_q8linear_backward(*a, **kw, want_dx=False, want_dw=False, want_dbias=True)[2], db.cpu(), "dbias alone")


def test_product_gradient_is_the_slope(dev):
    """Against differences of the forward pass's formula in 64 bits, along a random change of what the codes stand for."""
    say("product differences")
    rows, Cin, Cout = 40, 130, 70
    g = torch.Generator().manual_seed(3)
    xq, sx, wq, sw = make(g, rows, Cin, Cout)
    dy = torch.randn(rows, Cout, generator=g)
    p = q.Q8LinearPlan(rows, Cin, Cout, "gelu")
    bias = torch.randn(Cout, generator=g)
    y, z = q.wq8_q8linear_forward(p, *(t.to(dev) for t in (xq, sx, wq, sw, bias)), want_z=True)
    dx, dw, db = q.wq8_q8linear_backward(p, dy.to(dev), *(t.to(dev) for t in (xq, sx, wq, sw)), z=z, want_dbias=True)
    x, w, b = R.values(xq, sx, Cin), R.values(wq, sw, Cin), bias.double()
    vx, vw, vb = (torch.randn(t.shape, generator=g).double() for t in (x, w, b))
    eps = 1e-4  # its square times a third derivative, far below fp32's own roundings of z
    f = lambda s: (R.act((x + s * vx) @ (w + s * vw).T + b + s * vb, "gelu") * dy.double()).sum()  # noqa: E731
    diff = (f(eps) - f(-eps)) / (2 * eps)
    parts = [(d.cpu().double() * v) for d, v in ((dx, vx), (dw, vw), (db, vb))]
    dot, size = sum(t.sum() for t in parts), sum(t.abs().sum() for t in parts)
    assert abs(diff - dot) <= 1e-5 * size, (diff, dot)


def test_product_backward_borders(dev):
    """An infinity or a NaN in dy reaches its row of dx and its column's row of dw and dbias, nothing else."""
    say("product backward borders")
    for t in (F32, BF):
        rows, Cin, Cout = 140, 70, 40
        g = torch.Generator().manual_seed(5)
        xq, sx, wq, sw = make(g, rows, Cin, Cout)
        dy = torch.randn(rows, Cout, generator=g)
        clean = dy.clone()
        dy[3, 7], dy[130, 9] = float("inf"), float("nan")
        clean[3, 7], clean[130, 9] = 0, 0
        p = q.Q8LinearPlan(rows, Cin, Cout, x_dtype=t, y_dtype=F32)
        a = tuple(v.to(dev) for v in (xq, sx, wq, sw))
        dx, dw, db = (v.cpu().float() for v in q.wq8_q8linear_backward(p, dy.to(dev), *a, want_dbias=True))
        want = R.backward(clean, xq, sx, wq, sw, Cin, t)
        r, c = torch.ones(rows, dtype=torch.bool), torch.ones(Cout, dtype=torch.bool)
        r[[3, 130]], c[[7, 9]] = False, False
        assert torch.isnan(dx[~r]).all() and torch.isnan(dw[~c]).all() and not torch.isfinite(db[~c]).any()
        check(dx[r], want["dx"][0][r], want["dx"][1][r], "dx")
        check(dw[c], want["dw"][0][c], want["dw"][1][c], "dw")
        check(db[c], want["dbias"][0][c], want["dbias"][1][c], "dbias")
        # tiny gradients are no zeros
        small = clean * 2.0 ** -110
        dx, dw, _ = (v if v is None else v.cpu() for v in q.wq8_q8linear_backward(p, small.to(dev), *a))
        want = R.backward(small, xq, sx, wq, sw, Cin, t)
        check(dx, *want["dx"], "small dx")
        check(dw, *want["dw"], "small dw")


def test_no_rows(dev):
    say("no rows")
    e = lambda *s, t=F32: torch.empty(s, dtype=t, device=dev)  # noqa: E731
    p = q.QuantPlan(0, 40)
    assert q.wq8_quant_pack(p, e(0, 40))[0].shape == (0, 128)
    n = q.RmsPlan(0, 40)
    assert q.wq8_rms_forward(n, e(0, 40), want_codes=True)[2].shape == (0, 128)
    dx, dg = q.wq8_rms_backward(n, e(0, 40), e(0, 40), e(0), torch.ones(40, device=dev))
    assert dx.shape == (0, 40) and bool((dg == 0).all())
    for t in (F32, BF):
        m = q.Q8LinearPlan(0, 40, 50, x_dtype=t)
        w = (torch.ones(50, 128, dtype=torch.int8, device=dev), torch.ones(50, device=dev))
        x = (e(0, 128, t=torch.int8), e(0))
        assert q.wq8_q8linear_forward(m, *x, *w).shape == (0, 50)
        dx, dw, db = q.wq8_q8linear_backward(m, e(0, 50, t=t), *x, *w, want_dbias=True)
        assert dx.shape == (0, 40) and bool((dw == 0).all()) and bool((db == 0).all()) and dw.shape == (50, 40)
