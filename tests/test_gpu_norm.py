"""Group norm with an activation on the GPU against its definition in 64 bits:
both layouts, types, odd sizes, slices, the split and the fused schedules."""
import pytest
import torch

import ops_reference as R
import quantized_convolution_amd as q

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


def make(N, C, H, W, x_dtype, x_layout, seed, x_stride=0, affine=True, shift=False, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x = (r(N, H, W, C) * (1 + 0.3 * r(C)) + offset * r(C) + offset).to(x_dtype)
    x = x if x_layout == "nhwc" else x.permute(0, 3, 1, 2).contiguous()
    d = dict(x=x, gamma=1 + 0.2 * r(C) if affine else None, beta=0.2 * r(C) if affine else None,
             shift=r(N, C) if shift else None, dy=r(N, H, W, C))
    dev = {k: v.cuda() if v is not None else None for k, v in d.items()}
    if x_stride:
        wide = torch.full((N, H, W, x_stride), float("nan"), dtype=x_dtype, device="cuda")
        wide[..., :C] = dev["x"]
        dev["x"] = wide[..., :C]
    return d, dev


def run(N, C, H, W, groups, act, x_dtype=F32, y_dtype=F32, x_layout="nhwc", y_layout="nhwc", eps=1e-5, seed=0,
        x_stride=0, y_stride=0, affine=True, shift=False, backward=True, offset=0.5):
    print(f"[norm] N={N} C={C} {H}x{W} groups={groups} {act} {x_dtype}->{y_dtype} {x_layout}->{y_layout}", flush=True)
    d, dev = make(N, C, H, W, x_dtype, x_layout, seed, x_stride, affine, shift, offset)
    plan = q.NormPlan(N, C, H, W, groups=groups, eps=eps, act=act, x_dtype=x_dtype, y_dtype=y_dtype, x_layout=x_layout,
                      y_layout=y_layout, x_stride=x_stride, y_stride=y_stride)
    ref = R.Norm(R.nhwc(d["x"], x_layout), groups, eps, act, d["shift"], d["gamma"], d["beta"])
    y, mean, rstd = q.wq8_norm_forward(plan, dev["x"], dev["gamma"], dev["beta"], shift=dev["shift"], want_stats=True)
    torch.cuda.synchronize()
    em, er, ey = ref.forward_errors(y_dtype)
    R.check(mean, ref.mean, em + R.U * ref.mean.abs(), "mean")
    R.check(rstd, ref.rstd, er * ref.rstd, "rstd")
    R.check(R.nhwc(y, y_layout), ref.y, ey, "y")
    if not backward:
        return
    dy = d["dy"].to(y_dtype)
    dyl = dy if y_layout == "nhwc" else dy.permute(0, 3, 1, 2).contiguous()
    if y_stride:
        wide = torch.full((N, H, W, y_stride), float("nan"), dtype=y_dtype, device="cuda")
        wide[..., :C] = dyl.cuda()
        dyl = wide[..., :C]
    dx, dg, db, ds = q.wq8_norm_backward(plan, dyl.cuda(), dev["x"], ref.mean.float().cuda(), ref.rstd.float().cuda(),
                                         dev["gamma"], dev["beta"], shift=dev["shift"],
                                         dgamma=torch.empty(C, device="cuda"), dbeta=torch.empty(C, device="cuda"))
    torch.cuda.synchronize()
    want = ref.backward(dy, x_dtype)
    R.check(R.nhwc(dx, x_layout), *want["dx"], "dx")
    R.check(dg, *want["dgamma"], "dgamma")
    R.check(db, *want["dbeta"], "dbeta")
    assert (ds is None) == (not shift)
    if shift:
        R.check(ds, *want["dshift"], "dshift")


LAYOUTS = [("nhwc", "nhwc"), ("nchw", "nchw"), ("nhwc", "nchw"), ("nchw", "nhwc")]
TYPES = [(F32, F32), (BF, BF), (BF, F32), (F32, BF)]


# channels per group 1..80, odd ones among them; pixels from one to several blocks
@pytest.mark.parametrize("xl,yl", LAYOUTS)
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("C,H,W,groups", [(64, 7, 7, 32), (320, 16, 15, 32), (40, 9, 5, 8), (24, 33, 31, 8), (15, 17, 19, 3),
                                          (7, 8, 8, 1), (48, 1, 1, 3)])
def test_types_and_layouts(xl, yl, xt, yt, C, H, W, groups):
    run(2, C, H, W, groups, "silu", xt, yt, xl, yl, shift=True, seed=C)


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("xl,yl", LAYOUTS)
def test_activations(act, xl, yl):
    run(3, 64, 6, 11, 16, act, F32, F32, xl, yl, seed=5)


# groups too large for one block: split over the pixels, and over the channels of a group
@pytest.mark.parametrize("xl,yl", LAYOUTS)
@pytest.mark.parametrize("xt,yt", [(F32, F32), (BF, BF)])
@pytest.mark.parametrize("N,C,H,W,groups", [(1, 64, 128, 127, 2), (2, 2560, 8, 9, 1), (1, 1201, 9, 11, 1), (1, 33, 130, 129, 3),
                                            (1, 4, 301, 299, 1)])
def test_split(xl, yl, xt, yt, N, C, H, W, groups):
    run(N, C, H, W, groups, "silu", xt, yt, xl, yl, shift=True, seed=3)


@pytest.mark.parametrize("xl,yl", LAYOUTS)
@pytest.mark.parametrize("N,C,H,W,groups", [(1, 1, 1, 1, 1), (1, 8, 1, 1, 8), (5, 6, 1, 3, 2), (70, 3, 2, 2, 3), (1, 1, 300, 1, 1),
                                            (300, 32, 1, 2, 4)])
def test_smallest(xl, yl, N, C, H, W, groups):
    run(N, C, H, W, groups, "gelu", F32, F32, xl, yl, seed=8, eps=1e-3)


@pytest.mark.parametrize("xt", [F32, BF])
@pytest.mark.parametrize("extra", [1, 8, 40])
def test_slices(xt, extra):
    """Rows of a wider tensor: what lies beside them is NaN and is neither read nor written."""
    C = 40
    run(2, C, 9, 10, 8, "silu", xt, xt, x_stride=C + extra)
    run(2, C, 9, 10, 8, "silu", xt, xt, y_stride=C + extra)
    run(2, C, 9, 10, 8, "silu", xt, xt, "nchw", "nhwc", y_stride=C + extra)
    run(1, C, 90, 100, 2, "silu", xt, xt, x_stride=C + extra, y_stride=C + 2 * extra)
    _, dev = make(2, C, 9, 10, xt, "nhwc", 1)
    plan = q.NormPlan(2, C, 9, 10, groups=8, x_dtype=xt, y_stride=C + extra)
    wide = torch.full((2, 9, 10, C + extra), 7.0, dtype=xt, device="cuda")
    q.wq8_norm_forward(plan, dev["x"], y=wide[..., :C])
    torch.cuda.synchronize()
    assert (wide[..., C:] == 7).all()


def test_no_parameters():
    run(2, 32, 5, 6, 4, "relu", affine=False, seed=2)
    run(2, 32, 5, 6, 4, "none", affine=False, shift=True, seed=2)


@pytest.mark.parametrize("xl", ["nhwc", "nchw"])
@pytest.mark.parametrize("H", [16, 200])
def test_large_mean(xl, H):
    """A mean 300 times the deviation costs no more than its own rounding: squares are not subtracted."""
    run(1, 32, H, 16, 4, "none", x_layout=xl, y_layout=xl, offset=100.0, seed=4, backward=False)


def test_constant_group():
    """No deviation at all: rstd = 1 / sqrt(eps), y = act(beta)."""
    plan = q.NormPlan(2, 16, 4, 4, groups=4, eps=1e-6, act="silu")
    x = torch.full(plan.x_shape, 3.0, device="cuda")
    beta = torch.linspace(-2, 2, 16, device="cuda")
    y, mean, rstd = q.wq8_norm_forward(plan, x, None, beta, want_stats=True)
    torch.cuda.synchronize()
    assert (mean == 3).all() and torch.allclose(rstd, torch.full_like(rstd, 1e3), rtol=1e-6)
    R.check(y, R.act(beta.cpu().double(), "silu").expand(2, 4, 4, 16), 8 * R.U * 3, "y")


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("xl,yl", LAYOUTS)
@pytest.mark.parametrize("H", [6, 150])
def test_not_finite_stays_in_its_group(bad, xl, yl, H):
    _, dev = make(2, 16, H, 60, F32, xl, 1)
    R.nhwc(dev["x"], xl)[1, 2, 3, 5] = bad  # group 1 of image 1
    plan = q.NormPlan(2, 16, H, 60, groups=4, act="silu", x_layout=xl, y_layout=yl)
    y = R.nhwc(q.wq8_norm_forward(plan, dev["x"], dev["gamma"], dev["beta"]), yl)
    torch.cuda.synchronize()
    sick = torch.zeros(2, H, 60, 16, dtype=torch.bool)
    sick[1, :, :, 4:8] = True
    assert torch.isnan(y.cpu()[sick]).all() and torch.isfinite(y.cpu()[~sick]).all()


def test_empty_batch():
    plan = q.NormPlan(0, 8, 4, 4, groups=2)
    x = torch.empty(plan.x_shape, device="cuda")
    assert q.wq8_norm_forward(plan, x).shape == (0, 4, 4, 8)
    s = torch.empty((0, 2), device="cuda")
    g = torch.full((8,), 5.0, device="cuda")
    _, dg, db, _ = q.wq8_norm_backward(plan, x, x, s, s, g, g)
    torch.cuda.synchronize()
    assert (dg == 0).all() and (db == 0).all()


@pytest.mark.parametrize("xl,yl,H", [("nhwc", "nhwc", 16), ("nchw", "nhwc", 16), ("nhwc", "nhwc", 200)])
def test_gradient_against_differences(xl, yl, H):
    """d/dh of sum(y dy) along random directions, by central differences of the
    forward kernel: rounding leaves 3 U sqrt(n) |y dy| / h and the third
    derivative n h^2 / 6, n values of order one."""
    N, C, W, h = 1, 16, 16, 2.0 ** -6
    n = N * C * H * W
    d, dev = make(N, C, H, W, F32, xl, 11, shift=True)
    plan = q.NormPlan(N, C, H, W, groups=4, act="silu", x_layout=xl, y_layout=yl)
    dy = (d["dy"] if yl == "nhwc" else d["dy"].permute(0, 3, 1, 2).contiguous()).cuda()
    names = ("x", "gamma", "beta", "shift")

    def loss(a):
        y = q.wq8_norm_forward(plan, a["x"], a["gamma"], a["beta"], shift=a["shift"])
        return (y.double() * dy.double()).sum().item()

    _, mean, rstd = q.wq8_norm_forward(plan, dev["x"], dev["gamma"], dev["beta"], shift=dev["shift"], want_stats=True)
    grads = dict(zip(names, q.wq8_norm_backward(plan, dy, dev["x"], mean, rstd, dev["gamma"], dev["beta"], shift=dev["shift"])))
    g = torch.Generator().manual_seed(1)
    for k in names:
        v = torch.randn(dev[k].shape, generator=g).cuda()
        up, down = dict(dev, **{k: dev[k] + h * v}), dict(dev, **{k: dev[k] - h * v})
        diff = (loss(up) - loss(down)) / (2 * h)
        want = (grads[k].double() * v.double()).sum().item()
        spread = v.abs().max().item() ** 3
        tol = 10 * R.U * n ** 0.5 * 3 / h + spread * n * h * h / 6
        assert abs(diff - want) <= tol, (k, diff, want, tol)


def test_repeats_and_does_not_depend_on_the_workspace():
    """Same bits from every call, whatever the workspace held."""
    d, dev = make(2, 64, 100, 90, BF, "nhwc", 3)
    plan = q.NormPlan(2, 64, 100, 90, groups=2, act="silu", x_dtype=BF)
    dy = d["dy"].to(BF).cuda()
    got = []
    for fill in (0, 255, 127):
        ws = torch.full((plan.workspace_bytes,), fill, dtype=torch.uint8, device="cuda")
        wb = torch.full((plan.backward_workspace_bytes,), fill, dtype=torch.uint8, device="cuda")
        y, mean, rstd = q.wq8_norm_forward(plan, dev["x"], dev["gamma"], dev["beta"], want_stats=True, workspace=ws)
        dx, dg, db, _ = q.wq8_norm_backward(plan, dy, dev["x"], mean, rstd, dev["gamma"], dev["beta"], workspace=wb)
        got.append([t.clone() for t in (y, mean, rstd, dx, dg, db)])
    torch.cuda.synchronize()
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_offsets_past_32_bits():
    """A tensor of more than 2^32 bytes and 2^31 elements: the last image is right."""
    N, C, H, W = 9, 1024, 512, 512
    plan = q.NormPlan(N, C, H, W, groups=32, act="silu", x_dtype=BF)
    x = torch.zeros(plan.x_shape, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    x[-1] = torch.randn((H, W, C), generator=g, device="cuda", dtype=BF)
    y = q.wq8_norm_forward(plan, x)
    want = x[-1].double().reshape(H * W, 32, 32)
    want = (want - want.mean(dim=(0, 2), keepdim=True)) / torch.sqrt(want.var(dim=(0, 2), keepdim=True, correction=0) + 1e-5)
    want = want / (1 + torch.exp(-want))
    assert (y[:-1] == 0).all()
    off = (y[-1].double().reshape(H * W, 32, 32) - want).abs()
    assert (off <= R.BF16 * want.abs() + 2e-5).all()


def test_more_threads_than_one_grid_row_takes():
    """2^26 images of 4 values: more than 2^32 threads in each kernel. The last images are right."""
    N, C = (1 << 26) + 5, 4
    plan = q.NormPlan(N, C, 1, 1, groups=1, act="silu")
    x = torch.zeros(plan.x_shape, device="cuda")
    g = torch.Generator().manual_seed(6)
    last = torch.randn((9, 1, 1, C), generator=g)
    x[-9:] = last.cuda()
    y, mean, rstd = q.wq8_norm_forward(plan, x, want_stats=True)
    ref = R.Norm(last, 1, 1e-5, "silu")
    R.check(y[-9:], ref.y, ref.forward_errors(F32)[2], "y")
    assert torch.count_nonzero(y[:-9]) == 0 and torch.count_nonzero(mean[:-9]) == 0
    dy, shift = torch.ones_like(x), torch.zeros((N, C), device="cuda")
    dx, _, _, ds = q.wq8_norm_backward(plan, dy, x, mean, rstd, shift=shift)
    want = ref.backward(torch.ones(9, 1, 1, C), F32)
    R.check(dx[-9:], want["dx"][0], 2 * want["dx"][1], "dx")
    R.check(ds[-9:], want["dshift"][0], 2 * want["dshift"][1], "dshift")
    # x is 0 in the others: z = h = 0, dz the slope 1/2 of silu at 0, and dx what that leaves of its mean
    assert torch.count_nonzero(dx[:-9]) == 0 and torch.count_nonzero(ds[:-9]) == 0


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("xt", [F32, BF])
def test_fp32_activations(name, xt):
    """fp32 results have fp32 activations (bounds as for the product's)."""
    from test_gpu_linear import act_points, exact_acts

    z = act_points()[:5004].to(xt)
    n = len(z)
    # the backward takes mean and rstd: with 0 and 1, z is x itself and dbeta of one pixel the slope
    plan = q.NormPlan(1, n, 1, 1, groups=1, act=name, x_dtype=xt, y_dtype=F32)
    x, ones = z.reshape(plan.x_shape).cuda(), torch.ones(plan.y_shape, device="cuda")
    zero, one = torch.zeros(1, 1, device="cuda"), torch.ones(1, 1, device="cuda")
    _, slope, _, es = exact_acts(z, name)
    db = q.wq8_norm_backward(plan, ones, x, zero, one, dbeta=torch.empty(n, device="cuda"))[2]
    R.check(db, slope, es + 1e-37, "slope")
    # forward: z as the mean and rstd that it returns give it, to 6 U
    gamma, beta = torch.full((n,), 4.0, device="cuda"), torch.full((n,), -1.0, device="cuda")
    y, mean, rstd = q.wq8_norm_forward(plan, x, gamma, beta, want_stats=True)
    h = (z.double() - mean.cpu().double()) * rstd.cpu().double() * 4
    ez = 6 * R.U * (h.abs() + (mean.cpu().double() * rstd.cpu().double() * 4).abs() + 1)
    y64, slope, ey, _ = exact_acts((h - 1)[0], name)
    R.check(y.reshape(-1), y64, ey + 1.2 * ez[0] * slope.abs() + ez[0] ** 2 + 1e-37, "y")


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("xl,yl", LAYOUTS)
@pytest.mark.parametrize("C", [16, 24])
@pytest.mark.parametrize("H", [6, 150])
def test_statistics_of_what_is_not_finite(bad, xl, yl, C, H):
    """mean = sum v / m as the formula gives it, in one kernel and split over two: an infinity
    among finite values is the mean, two of opposite sign or a NaN make a NaN; rstd is a NaN."""
    _, dev = make(2, C, H, 60, F32, xl, 1)
    x = R.nhwc(dev["x"], xl)
    w = C // 4
    x[1, 2, 3, w + 1] = bad                                                  # group 1 of image 1
    x[0, H - 1, 59, C - 1], x[0, 0, 0, C - 2] = bad, -bad                    # group 3 of image 0
    x[0, 0, 0, 0] = bad                                                      # the first value of a block
    plan = q.NormPlan(2, C, H, 60, groups=4, act="silu", x_layout=xl, y_layout=yl)
    _, mean, rstd = q.wq8_norm_forward(plan, dev["x"], dev["gamma"], dev["beta"], want_stats=True)
    torch.cuda.synchronize()
    want = torch.tensor(bad)
    for n, g in ((1, 1), (0, 0)):
        assert torch.equal(mean[n, g].cpu(), want) or (torch.isnan(want) and torch.isnan(mean[n, g])), (n, g, mean)
    assert torch.isnan(mean[0, 3])
    sick = torch.zeros(2, 4, dtype=torch.bool)
    sick[1, 1] = sick[0, 0] = sick[0, 3] = True
    assert torch.isnan(rstd.cpu()[sick]).all()
    assert torch.isfinite(mean.cpu()[~sick]).all() and torch.isfinite(rstd.cpu()[~sick]).all()


@pytest.mark.parametrize("xl,yl", LAYOUTS)
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("H,C,groups", [(5, 512, 32), (5, 480, 32), (140, 480, 4)])
def test_relu_has_one_mask(xl, yl, xt, yt, H, C, groups):
    """The backward's relu passes exactly where the forward's did. beta puts z of one pixel within rounding of 0
    in every channel; dy is 1 there and 0 elsewhere, so that dbeta is the mask of the backward."""
    W = 31
    _, dev = make(1, C, H, W, xt, xl, 21)
    plan = q.NormPlan(1, C, H, W, groups=groups, act="relu", x_dtype=xt, y_dtype=yt, x_layout=xl, y_layout=yl)
    gamma = dev["gamma"]
    _, mean, rstd = q.wq8_norm_forward(plan, dev["x"], want_stats=True)
    x = R.nhwc(dev["x"], xl)[0, 2, 7].double()
    spread = lambda s: s[0].double().repeat_interleave(C // groups)  # noqa: E731
    beta = -((x - spread(mean)) * spread(rstd) * gamma.double()).float()
    y, m2, r2 = q.wq8_norm_forward(plan, dev["x"], gamma, beta, want_stats=True)
    assert torch.equal(m2, mean) and torch.equal(r2, rstd)
    dy = torch.zeros(plan.y_shape, dtype=yt, device="cuda")
    R.nhwc(dy, yl)[0, 2, 7] = 1
    db = q.wq8_norm_backward(plan, dy, dev["x"], mean, rstd, gamma, beta)[2]
    mask = (R.nhwc(y, yl)[0, 2, 7] > 0).float()
    assert 0 < mask.sum() < C
    assert torch.equal(db, mask)
