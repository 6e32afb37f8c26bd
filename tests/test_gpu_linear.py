"""Matrix product with bias, activation and residual on the GPU against its
definition in 64 bits: types, odd sizes, slices, residual layouts, gradients."""
import pytest
import torch

import ops_reference as R
import quantized_convolution_amd as q

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


def strided(t, extra):
    """`t` on the GPU in rows of a wider tensor whose other columns are NaN."""
    if not extra:
        return t.cuda()
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t.cuda()
    return wide[:, :t.shape[1]]


def make(rows, Cin, Cout, xt, yt, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(x=r(rows, Cin).to(xt), w=(r(Cout, Cin) / Cin ** 0.5).to(xt), bias=0.5 * r(Cout), res=r(rows, Cout).to(yt),
                dy=r(rows, Cout).to(yt))


def forward(rows, Cin, Cout, act="none", xt=F32, yt=F32, bias=True, residual="none", pixels=0, want_z=False, sx=0, sy=0, sr=0,
            seed=0):
    print(f"[linear] {rows}x{Cin}x{Cout} {act} {xt}->{yt} residual={residual} strides +{sx} +{sy} +{sr}", flush=True)
    d = make(rows, Cin, Cout, xt, yt, seed)
    planar = residual == "planar"
    plan = q.LinearPlan(rows, Cin, Cout, act=act, x_dtype=xt, y_dtype=yt, r_layout="nchw" if planar else "nhwc", pixels=pixels,
                        x_stride=Cin + sx if sx else 0, y_stride=Cout + sy if sy else 0, r_stride=Cout + sr if sr else 0)
    res = None
    if residual == "rows":
        res = strided(d["res"], sr)
    elif planar:
        res = d["res"].reshape(rows // pixels, pixels, Cout).permute(0, 2, 1).contiguous().cuda()
    y = strided(torch.zeros(rows, Cout, dtype=yt), sy)
    z = torch.empty(rows, Cout, dtype=yt, device="cuda") if want_z else None
    q.wq8_linear_forward(plan, strided(d["x"], sx), d["w"].cuda(), d["bias"].cuda() if bias else None, res, y=y, z=z)
    torch.cuda.synchronize()
    ry, rz = R.linear_forward(d["x"], d["w"], d["bias"] if bias else None, d["res"] if residual != "none" else None, act, yt)
    R.check(y, *ry, "y")
    if want_z:
        R.check(z, *rz, "z")
    if sy:  # what lies beside the slice is untouched
        assert torch.isnan(y.as_strided((rows, sy), (Cout + sy, 1), Cout)).all()


def backward(rows, Cin, Cout, act="none", xt=F32, yt=F32, sx=0, sy=0, seed=0):
    print(f"[linear backward] {rows}x{Cin}x{Cout} {act} {xt}->{yt} strides +{sx} +{sy}", flush=True)
    d = make(rows, Cin, Cout, xt, yt, seed)
    z = (d["x"].double() @ d["w"].double().T + d["bias"].double()).to(yt)
    plan = q.LinearPlan(rows, Cin, Cout, act=act, x_dtype=xt, y_dtype=yt, x_stride=Cin + sx if sx else 0,
                        y_stride=Cout + sy if sy else 0)
    dx = strided(torch.zeros(rows, Cin, dtype=xt), sx)
    _, dw, db = q.wq8_linear_backward(plan, strided(d["dy"], sy), strided(d["x"], sx), d["w"].cuda(), z=z.cuda(), dx=dx,
                                      want_dbias=True)
    torch.cuda.synchronize()
    want = R.linear_backward(d["dy"], d["x"], d["w"], z, act, xt, xt == BF and (act != "none" or yt != BF))
    R.check(dx, *want["dx"], "dx")
    R.check(dw, *want["dw"], "dw")
    R.check(db, *want["dbias"], "dbias")


TYPES = [(F32, F32), (BF, BF), (BF, F32), (F32, BF)]
# one row, one column, one k, odd ones, tile edges on either side, several tiles
SIZES = [(1, 1, 1), (1, 64, 64), (3, 5, 7), (8, 320, 200), (16, 33, 130), (17, 129, 31), (65, 64, 127), (128, 72, 128), (129, 200, 257),
         (300, 515, 129), (64, 1000, 48)]


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("size", SIZES)
def test_forward_sizes(xt, yt, size):
    forward(*size, "none", xt, yt)
    forward(*size, "silu", xt, yt, residual="rows", want_z=True, seed=1)


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("size", SIZES)
def test_backward_sizes(xt, yt, size):
    backward(*size, "none", xt, yt)
    backward(*size, "silu", xt, yt, seed=1)


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("xt", [F32, BF])
def test_activations(act, xt):
    forward(70, 96, 90, act, xt, xt, want_z=True, seed=2)
    forward(70, 96, 90, act, xt, xt, bias=False, residual="rows", seed=3)
    backward(70, 96, 90, act, xt, xt, seed=2)


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("images,pixels,Cout", [(1, 1, 5), (3, 49, 64), (2, 256, 72), (5, 7, 33), (200, 1, 130)])
def test_planar_residual(xt, yt, images, pixels, Cout):
    forward(images * pixels, 40, Cout, "gelu", xt, yt, residual="planar", pixels=pixels, seed=4)


@pytest.mark.parametrize("xt", [F32, BF])
@pytest.mark.parametrize("extra", [1, 4, 8, 56])
def test_slices(xt, extra):
    for size in ((37, 72, 50), (130, 128, 136), (4, 128, 96)):
        forward(*size, "silu", xt, xt, residual="rows", sx=extra, sy=extra, sr=extra, seed=5)
        backward(*size, "silu", xt, xt, sx=extra, sy=extra, seed=5)
        backward(*size, "none", xt, xt, sx=extra, sy=extra, seed=6)


# few tiles and a long sum: k is split over blocks and joined
@pytest.mark.parametrize("xt", [F32, BF])
@pytest.mark.parametrize("size", [(20, 4100, 24), (100, 2050, 130), (4100, 40, 50), (2500, 130, 100), (33, 64, 5000)])
def test_long_sums(xt, size):
    forward(*size, "gelu", xt, xt, residual="rows", want_z=True, seed=7)
    backward(*size, "gelu_tanh", xt, xt, seed=7)


def test_residual_in_place():
    d = make(70, 64, 40, F32, F32, 3)
    plan = q.LinearPlan(70, 64, 40)
    y = d["res"].cuda()
    q.wq8_linear_forward(plan, d["x"].cuda(), d["w"].cuda(), d["bias"].cuda(), y, y=y)
    torch.cuda.synchronize()
    R.check(y, *R.linear_forward(d["x"], d["w"], d["bias"], d["res"], "none", F32)[0], "y")


@pytest.mark.parametrize("xt", [F32, BF])
def test_only_what_is_wanted(xt):
    d = make(70, 64, 40, xt, xt, 3)
    plan = q.LinearPlan(70, 64, 40, x_dtype=xt)
    a = (plan, d["dy"].cuda(), d["x"].cuda(), d["w"].cuda())
    full = q.wq8_linear_backward(*a, want_dbias=True)
    for k in range(3):
        wants = dict(want_dx=k == 0, want_dw=k == 1, want_dbias=k == 2)
        got = q.wq8_linear_backward(*a, **wants)
        torch.cuda.synchronize()
        assert [g is not None for g in got] == [k == i for i in range(3)]
        assert torch.equal(got[k], full[k])


def test_no_rows():
    plan = q.LinearPlan(0, 16, 8, act="silu")
    x, dy, w = torch.empty(0, 16, device="cuda"), torch.empty(0, 8, device="cuda"), torch.ones(8, 16, device="cuda")
    assert q.wq8_linear_forward(plan, x, w).shape == (0, 8)
    dx, dw, db = q.wq8_linear_backward(plan, dy, x, w, z=dy, dw=torch.ones_like(w), dbias=torch.ones(8, device="cuda"))
    torch.cuda.synchronize()
    assert dx.shape == (0, 16) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("xt", [F32, BF])
@pytest.mark.parametrize("rows", [4, 150])
def test_not_finite_stays_in_its_row(xt, rows):
    """What is added to fill a tile must not meet an infinity: 0 * inf is NaN."""
    for Cin in (72, 77):
        d = make(rows, Cin, 90, xt, xt, 5)
        d["x"][2, 5], d["x"][3, Cin - 1] = float("inf"), float("nan")
        plan = q.LinearPlan(rows, Cin, 90, act="none", x_dtype=xt)
        y = q.wq8_linear_forward(plan, d["x"].cuda(), d["w"].cuda(), d["bias"].cuda())
        torch.cuda.synchronize()
        y = y.cpu().float()
        fine = torch.ones(rows, dtype=torch.bool)
        fine[2:4] = False
        assert torch.isfinite(y[fine]).all()
        assert (y[2] == torch.sign(d["w"][:, 5].float()) * float("inf")).all() and torch.isnan(y[3]).all()


def test_relu_keeps_nan():
    d = make(4, 8, 4, F32, F32, 1)
    d["x"][1, 1] = float("nan")
    y = q.wq8_linear_forward(q.LinearPlan(4, 8, 4, act="relu"), d["x"].cuda(), d["w"].cuda())
    torch.cuda.synchronize()
    assert torch.isnan(y[1]).all() and (y[[0, 2, 3]] >= 0).all()


def test_gradient_against_differences():
    """Central differences of the forward along random directions (see the
    group norm's): z along a direction moves by sums of Cin terms of order
    h / sqrt(Cin), and the loss sums n values."""
    rows, Cin, Cout, h = 40, 24, 36, 2.0 ** -6
    n = rows * Cout
    d = {k: v.cuda() for k, v in make(rows, Cin, Cout, F32, F32, 9).items()}
    plan = q.LinearPlan(rows, Cin, Cout, act="gelu")
    names = ("x", "w", "bias")

    def loss(a):
        y = q.wq8_linear_forward(plan, a["x"], a["w"], a["bias"], a["res"])
        return (y.double() * d["dy"].double()).sum().item()

    _, z = q.wq8_linear_forward(plan, d["x"], d["w"], d["bias"], d["res"], want_z=True)
    grads = dict(zip(names, q.wq8_linear_backward(plan, d["dy"], d["x"], d["w"], z=z, want_dbias=True)))
    g = torch.Generator().manual_seed(1)
    for k in names:
        v = torch.randn(d[k].shape, generator=g).cuda()
        if k == "w":
            v /= Cin ** 0.5
        up, down = dict(d, **{k: d[k] + h * v}), dict(d, **{k: d[k] - h * v})
        diff = (loss(up) - loss(down)) / (2 * h)
        want = (grads[k].double() * v.double()).sum().item()
        tol = 10 * R.U * n ** 0.5 * 3 / h + 4 ** 3 * n * h * h / 6
        assert abs(diff - want) <= tol, (k, diff, want, tol)


@pytest.mark.parametrize("xt", [F32, BF])
def test_repeats_and_does_not_depend_on_the_workspace(xt):
    rows, Cin, Cout = 300, 2100, 70
    d = {k: v.cuda() for k, v in make(rows, Cin, Cout, xt, xt, 9).items()}
    plan = q.LinearPlan(rows, Cin, Cout, act="silu", x_dtype=xt)
    got = []
    for fill in (0, 255, 127):
        ws = torch.full((plan.workspace_bytes,), fill, dtype=torch.uint8, device="cuda")
        wb = torch.full((plan.backward_workspace_bytes,), fill, dtype=torch.uint8, device="cuda")
        y, z = q.wq8_linear_forward(plan, d["x"], d["w"], d["bias"], d["res"], want_z=True, workspace=ws)
        g = q.wq8_linear_backward(plan, d["dy"], d["x"], d["w"], z=z, want_dbias=True, workspace=wb)
        got.append([t.clone() for t in (y, z, *g)])
    torch.cuda.synchronize()
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_offsets_past_32_bits():
    """x of more than 2^32 bytes and 2^31 elements, y too: the last rows are right, in both directions."""
    rows, Cin, Cout = 2 ** 20 + 65, 2056, 2064
    x = torch.zeros((rows, Cin), dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    x[-3:] = torch.randn((3, Cin), generator=g, device="cuda", dtype=BF)
    w = (torch.randn((Cout, Cin), generator=g, device="cuda") / Cin ** 0.5).to(BF)
    plan = q.LinearPlan(rows, Cin, Cout, x_dtype=BF)
    y = q.wq8_linear_forward(plan, x, w)
    R.check(y[-3:], *R.linear_forward(x[-3:].cpu(), w.cpu(), None, None, "none", BF)[0], "y")
    assert (y[:-3] == 0).all()
    dy = y  # as good as any
    dx, dw, _ = q.wq8_linear_backward(plan, dy, x, w)
    want = R.linear_backward(dy[-3:].cpu(), x[-3:].cpu(), w.cpu(), None, "none", BF, False)
    R.check(dx[-3:], *want["dx"], "dx")
    R.check(dw, *want["dw"], "dw")
    assert (dx[:-3] == 0).all()


@pytest.mark.parametrize("act,yt", [("silu", BF), ("gelu", F32), ("none", F32)])
@pytest.mark.parametrize("size", [(1, 40, 24), (9, 65, 130), (40, 16, 100), (300, 70, 33), (5, 700, 129), (1100, 24, 31)])
def test_few_values_keep_what_rounding_leaves(act, yt, size):
    """With few values dz goes into the bf16 products as two matrices: to 16 bits,
    so that the final rounding is all that is left beside fp32 arithmetic."""
    rows, Cin, Cout = size
    d = make(rows, Cin, Cout, BF, yt, 12)
    z = (d["x"].double() @ d["w"].double().T + d["bias"].double()).to(yt)
    plan = q.LinearPlan(rows, Cin, Cout, act=act, x_dtype=BF, y_dtype=yt)
    got = q.wq8_linear_backward(plan, d["dy"].cuda(), d["x"].cuda(), d["w"].cuda(), z=z.cuda(), want_dbias=True)
    torch.cuda.synchronize()
    want = R.linear_backward(d["dy"], d["x"], d["w"], z, act, BF, False)
    dz = d["dy"].double().abs() * (R.slope(z.double(), act).abs() + 1e-6) if act != "none" else d["dy"].double().abs()
    rest = 2.0 ** -16 * dz  # rounding of the second matrix
    R.check(got[0], want["dx"][0], want["dx"][1] + 1.01 * (rest @ d["w"].double().abs()), "dx")
    R.check(got[1], want["dw"][0], want["dw"][1] + 1.01 * (rest.T @ d["x"].double().abs()), "dw")
    R.check(got[2], *want["dbias"], "dbias")


@pytest.mark.parametrize("size", [(600, 300, 400), (520, 264, 328)])
@pytest.mark.parametrize("act,yt", [("silu", BF), ("none", F32)])
def test_many_values(size, act, yt):
    backward(*size, act, BF, yt, seed=13)


def dz_bounds(d, z, act, want):
    """`want` of linear_backward without a rounding of dz, and what two bf16
    matrices leave of dz: each value cut after 8 bits and the rest rounded to 8
    more, 2^-16 of it at most."""
    dz = d["dy"].double().abs() * (R.slope(z.double(), act).abs() + 1e-6)
    rest = 1.01 * 2.0 ** -16 * dz
    return {"dx": (want["dx"][0], want["dx"][1] + rest @ d["w"].double().abs()),
            "dw": (want["dw"][0], want["dw"][1] + rest.T @ d["x"].double().abs()), "dbias": want["dbias"]}


@pytest.mark.parametrize("act,yt", [("silu", BF), ("gelu", F32), ("none", F32)])
@pytest.mark.parametrize("size", [(600, 300, 400), (520, 264, 328), (1100, 2100, 136), (2000, 72, 1024)])
def test_many_values_keep_what_rounding_leaves(act, yt, size):
    """As with few values: the precision of dx and dw does not depend on the size."""
    rows, Cin, Cout = size
    d = make(rows, Cin, Cout, BF, yt, 14)
    z = (d["x"].double() @ d["w"].double().T + d["bias"].double()).to(yt)
    plan = q.LinearPlan(rows, Cin, Cout, act=act, x_dtype=BF, y_dtype=yt)
    got = q.wq8_linear_backward(plan, d["dy"].cuda(), d["x"].cuda(), d["w"].cuda(), z=z.cuda(), want_dbias=True)
    torch.cuda.synchronize()
    want = dz_bounds(d, z, act, R.linear_backward(d["dy"], d["x"], d["w"], z, act, BF, False))
    for t, k in zip(got, want):
        R.check(t, *want[k], k)


@pytest.mark.parametrize("size", [(20, 40, 24), (600, 300, 400)])
def test_backward_infinities(size):
    """An infinity in w or x meets every value of dz that is not zero with that
    value's sign, however dz is held: no NaN in place of an infinity. Where dz is
    zero the product is a NaN."""
    rows, Cin, Cout = size
    d = make(rows, Cin, Cout, BF, F32, 15)
    d["dy"][::3] = d["dy"][::3].to(BF).float()  # nothing is left by rounding
    d["dy"][1, 4], d["dy"][5, 4] = 0.0, -0.0
    d["w"][4, 7], d["x"][2, 9] = float("inf"), float("-inf")
    plan = q.LinearPlan(rows, Cin, Cout, x_dtype=BF, y_dtype=F32)
    dx, dw, _ = q.wq8_linear_backward(plan, d["dy"].cuda(), d["x"].cuda(), d["w"].cuda())
    torch.cuda.synchronize()
    dx, dw = dx.cpu().float(), dw.cpu().float()
    zero = d["dy"][:, 4] == 0
    assert torch.isnan(dx[zero, 7]).all()
    assert torch.equal(dx[~zero, 7], torch.sign(d["dy"][~zero, 4]) * float("inf"))
    assert torch.isfinite(dx[:, :7]).all() and torch.isfinite(dx[:, 8:]).all()
    assert torch.equal(dw[:, 9], torch.sign(d["dy"][2]) * float("-inf"))
    assert torch.isfinite(dw[:, :9]).all() and torch.isfinite(dw[:, 10:]).all()


@pytest.mark.parametrize("act,yt", [("silu", BF), ("none", F32)])
@pytest.mark.parametrize("size", [(40, 65, 130), (600, 300, 400)])
def test_rounded_dz(act, yt, size):
    """A caller may have dz rounded to bf16 in the products; everything else stays as it is."""
    rows, Cin, Cout = size
    d = make(rows, Cin, Cout, BF, yt, 16)
    z = (d["x"].double() @ d["w"].double().T + d["bias"].double()).to(yt)
    plans = [q.LinearPlan(rows, Cin, Cout, act=act, x_dtype=BF, y_dtype=yt, round_dz=r) for r in (False, True)]
    a = [d[k].cuda() for k in ("dy", "x", "w")]
    exact, got = (q.wq8_linear_backward(p, *a, z=z.cuda(), want_dbias=True) for p in plans)
    torch.cuda.synchronize()
    want = R.linear_backward(d["dy"], d["x"], d["w"], z, act, BF, True)
    for t, k in zip(got, want):
        R.check(t, *want[k], k)
    assert torch.equal(got[2], exact[2]) and not torch.equal(got[0], exact[0])
    assert plans[1].backward_workspace_bytes < plans[0].backward_workspace_bytes


def test_more_threads_than_one_grid_row_takes():
    """2^30 rows: more than 2^32 threads in each kernel. The last rows are right in both directions, and
    the sums over all of them: powers of two and few values that are not zero, exact in any order."""
    rows, Cin, Cout = (1 << 30) + 65, 4, 4
    x, dy = (torch.zeros((rows, Cin), dtype=BF, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(4)
    some = torch.cat([torch.arange(3), torch.arange(rows // 2, rows // 2 + 3), torch.arange(rows - 70, rows)]).cuda()
    draw = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").to(BF)  # noqa: E731
    x[some], dy[some], w = draw(len(some), Cin), draw(len(some), Cout), draw(Cout, Cin)
    plan = q.LinearPlan(rows, Cin, Cout, act="relu", x_dtype=BF)
    y, z = q.wq8_linear_forward(plan, x, w, want_z=True)
    want = x[some].double() @ w.double().T
    assert torch.equal(z[some].double(), want) and torch.equal(y[some].double(), want.clamp(min=0))
    assert torch.count_nonzero(y) == torch.count_nonzero(want > 0)
    del y
    dx, dw, db = q.wq8_linear_backward(plan, dy, x, w, z=z, want_dbias=True)
    dz = dy[some].double() * (want > 0)
    off = dx[some].double() - dz @ w.double()
    assert off.abs().max().item() <= 1e-35 and torch.count_nonzero(dx.view(torch.int16)[8:rows // 2 - 8] & 0x7f80) == 0
    assert (dw.double() - dz.T @ x[some].double()).abs().max().item() <= 1e-35
    assert torch.equal(db.double(), dz.sum(0))


def exact_acts(z, name):
    """(act, its slope, bounds of both) of fp32 values in 64 bits, for arithmetic
    in fp32 throughout: a few roundings relative to the terms that are summed.
    s, the gate: exp and reciprocal to one unit in the last place each (2 U), its
    argument rounded as the formula has it; the sum, the products: U each."""
    z = z.double()
    if name == "silu":
        s, rel = 1 / (1 + torch.exp(-z)), 8.0
        return z * s, R.slope(z, name), rel * R.U * (z * s).abs(), 12 * R.U * s * (1 + z.abs())
    if name == "gelu":
        # the fit and its sum 12 U, the normal density 3, products
        cdf = 0.5 * torch.erfc(-z / 2 ** 0.5)
        pdf = torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
        return z * cdf, cdf + z * pdf, 20 * R.U * (z * cdf).abs(), 20 * R.U * (cdf + z.abs() * pdf)
    k, c = 2 * (2 / torch.pi) ** 0.5, 0.044715
    u = k * (z + c * z ** 3)
    s, w, rel = 1 / (1 + torch.exp(-u)), k * (1 + 3 * c * z * z), 8 + 6 * u.abs()
    p = z.abs() * s / (1 + torch.exp(u)) * w
    return (z * s, s + z * s / (1 + torch.exp(u)) * w, rel * R.U * (z * s).abs(),
            R.U * (rel * (s + p) + 4 * z.abs() * w * s))


def act_points():
    z = torch.cat([torch.linspace(-13, 13, 5000), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-3, -1e-3, 40.0, -40.0, 100.0, -100.0, 1e4, -1e4])])
    return z.float()


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_fp32_activations(name):
    """fp32 results have fp32 activations, whatever the inputs' type: one column, so that z is x itself."""
    z = act_points()
    y, slope, ey, es = exact_acts(z, name)
    plan = q.LinearPlan(len(z), 1, 1, act=name)
    one = torch.ones(1, 1, device="cuda")
    R.check(q.wq8_linear_forward(plan, z[:, None].cuda(), one)[:, 0], y, ey + 1e-37, "y")
    row = q.LinearPlan(1, 1, len(z), act=name)
    ones = torch.ones(1, len(z), device="cuda")
    db = q.wq8_linear_backward(row, ones, one, ones.T.contiguous(), z=z[None].cuda(), want_dbias=True)[2]
    R.check(db, slope, es + 1e-37, "slope")
    zb = z.to(BF)
    y, slope, ey, es = exact_acts(zb, name)
    plan = q.LinearPlan(len(z), 1, 1, act=name, x_dtype=BF, y_dtype=F32)
    R.check(q.wq8_linear_forward(plan, zb[:, None].cuda(), one.to(BF))[:, 0], y, ey + 1e-37, "y of bf16")
    row = q.LinearPlan(1, 1, len(z), act=name, x_dtype=F32, y_dtype=BF)
    db = q.wq8_linear_backward(row, ones.to(BF), one, ones.T.contiguous(), z=zb[None].cuda(), want_dbias=True)[2]
    R.check(db, slope, es + 1e-37, "slope of bf16")


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_activations_of_large_values(name, xt, yt):
    """Finite values whose powers are not: act(z) is z or 0, its slope 1 or 0, to the ends of the type."""
    z = torch.cat([s * 10.0 ** torch.arange(3, 38) for s in (1.0, -1.0)]).to(yt)
    n = len(z)
    one = torch.ones(1, 1, device="cuda")
    x = z.to(xt)
    y = q.wq8_linear_forward(q.LinearPlan(n, 1, 1, act=name, x_dtype=xt, y_dtype=yt), x[:, None].cuda(), one.to(xt))
    assert torch.equal(y[:, 0].cpu(), x.to(yt).clamp(min=0))
    row = q.LinearPlan(1, 1, n, act=name, x_dtype=xt, y_dtype=yt)
    dy = torch.full((1, n), 3.0, device="cuda", dtype=yt)
    dx, dw, db = q.wq8_linear_backward(row, dy, one.to(xt), torch.ones(n, 1, device="cuda", dtype=xt), z=z[None].cuda(),
                                       want_dbias=True)
    want = 3.0 * (z > 0)
    assert torch.equal(db.cpu(), want.float()) and torch.equal(dw[:, 0].cpu().float(), want.float())
    assert dx.item() == want.sum().item()


@pytest.mark.parametrize("round_dz", [False, True])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_backward_of_gradients_that_are_not_finite(bad, round_dz):
    """An infinity in dy is one in its row of dx and its row of dw with the sign of what it meets, and nowhere else."""
    d = make(40, 48, 56, BF, F32, 17)
    d["dy"][3, 5] = bad
    plan = q.LinearPlan(40, 48, 56, x_dtype=BF, y_dtype=F32, round_dz=round_dz)
    dx, dw, db = q.wq8_linear_backward(plan, d["dy"].cuda(), d["x"].cuda(), d["w"].cuda(), want_dbias=True)
    torch.cuda.synchronize()
    for got, row, other in ((dx, 3, d["w"][5]), (dw, 5, d["x"][3])):
        got = got.cpu().float()
        want = torch.sign(other.float()) * bad
        assert torch.equal(got[row].nan_to_num(7), want.nan_to_num(7))
        got[row] = 0
        assert torch.isfinite(got).all()
    assert torch.equal(db.cpu()[5].nan_to_num(7), torch.tensor(bad).nan_to_num(7)) and torch.isfinite(db).sum() == 55
