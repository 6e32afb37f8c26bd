"""Every kernel instance that the plans choose (plan_cases.py), on the GPU: the
product on whole numbers, where every sum is exact and a term that is lost, met
twice or out of place is a wrong number; the group norm against its definition
in 64 bits."""
import pytest
import torch

import ops_reference as R
import plan_cases as P
import quantized_convolution_amd as q

pytestmark = pytest.mark.gpu
TYPES = (torch.float32, torch.bfloat16)
LAYOUTS = ("nhwc", "nchw")


def whole(g, *shape, most=2):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int8)


def same(got, want, what):
    """Equal to the exact value, rounded to the result's type once."""
    want = want.to(got.dtype)
    off = got != want
    assert not off.any(), f"{what}: {int(off.sum())} of {off.numel()} values differ, first at {off.nonzero()[0].tolist()}"


@pytest.mark.parametrize("case", P.LINEAR, ids=lambda c: "x".join(map(str, c)))
def test_linear(case):
    rows, Cin, Cout, act, xt, yt, round_dz = case
    print(f"[linear plan] {case}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows)
    name, xt, yt = ("none", "relu")[act], TYPES[xt], TYPES[yt]
    x, w, dy, res, z = whole(g, rows, Cin), whole(g, Cout, Cin), whole(g, rows, Cout), whole(g, rows, Cout, most=9), whole(g, rows, Cout)
    bias = whole(g, Cout, most=9).float()
    assert 4 * max(Cin, Cout, rows) + 18 < 2 ** 24  # any partial sum is exact in fp32
    xd, wd = x.to(xt), w.to(xt)
    z64 = x.double() @ w.double().T + bias.double()
    y64 = z64.clamp(min=0) if act else z64
    pixels = next(p for p in [*range(2, 400), rows] if rows % p == 0)
    for planar in (False, True):
        for t in TYPES:
            plan = q.LinearPlan(rows, Cin, Cout, act=name, x_dtype=xt, y_dtype=t, r_layout=LAYOUTS[planar], pixels=pixels if planar else 0)
            r = res.reshape(-1, pixels, Cout).permute(0, 2, 1).contiguous() if planar else res
            y, zo = q.wq8_linear_forward(plan, xd, wd, bias, r.to(t), want_z=True)
            same(y, y64 + res, f"y {t} {LAYOUTS[planar]}")
            same(zo, z64, f"z {t}")
            del y, zo, r
    y = q.wq8_linear_forward(q.LinearPlan(rows, Cin, Cout, act=name, x_dtype=xt, y_dtype=yt), xd, wd)
    y64 = z64 - bias
    same(y, y64.clamp(min=0) if act else y64, "y alone")
    del y, y64, z64, res
    dz = dy.double() * (z > 0) if act else dy.double()
    plan = q.LinearPlan(rows, Cin, Cout, act=name, x_dtype=xt, y_dtype=yt, round_dz=bool(round_dz))
    got = q.wq8_linear_backward(plan, dy.to(yt), xd, wd, z=z.to(yt), want_dbias=True)
    same(got[0], dz @ w.double(), "dx")
    same(got[1], dz.T @ x.double(), "dw")
    same(got[2], dz.sum(0), "dbias")


def within(got, want, bound, what):
    off = (got.double() - want).abs()
    assert not torch.isnan(off).any(), f"{what}: NaN"
    worst = (off - bound).max().item()
    assert worst <= 0, f"{what}: off by {off.max().item():.3e}, {worst:.3e} over its bound"


def norm(case, acts):
    N, C, H, W, groups, xt, yt, xl, yl = case
    xt, yt, xl, yl = TYPES[xt], TYPES[yt], LAYOUTS[xl], LAYOUTS[yl]
    g = torch.Generator(device="cuda").manual_seed(C + N)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    to = lambda t, layout: t if layout == "nhwc" else t.permute(0, 3, 1, 2).contiguous()  # noqa: E731
    x = to(r(N, H, W, C) * (1 + 0.3 * r(C)) + 0.5 * r(C) + 0.5, xl).to(xt)
    gamma, beta, shift, dy = 1 + 0.2 * r(C), 0.2 * r(C), r(N, C), r(N, H, W, C).to(yt)
    dyl = to(dy, yl)
    for act in acts:
        print(f"[norm plan] {case} {act}", flush=True)
        plan = q.NormPlan(N, C, H, W, groups=groups, eps=1e-5, act=act, x_dtype=xt, y_dtype=yt, x_layout=xl, y_layout=yl)
        ref = R.Norm(R.nhwc(x, xl), groups, 1e-5, act, shift, gamma, beta)
        y, dx = plan.empty_output().fill_(float("nan")), plan.empty_input().fill_(float("nan"))
        _, mean, rstd = q.wq8_norm_forward(plan, x, gamma, beta, shift=shift, y=y, want_stats=True)
        em, er, ey = ref.forward_errors(yt)
        within(mean, ref.mean, em + R.U * ref.mean.abs(), "mean")
        within(rstd, ref.rstd, er * ref.rstd, "rstd")
        within(R.nhwc(y, yl), ref.y, ey, "y")
        del y, ey
        if act == "relu":  # its gradient jumps within the rounding of z
            continue
        got = q.wq8_norm_backward(plan, dyl, x, ref.mean.float(), ref.rstd.float(), gamma, beta, shift=shift, dx=dx)
        want = ref.backward(dy, xt)
        within(R.nhwc(got[0], xl), *want["dx"], "dx")
        for t, k in zip(got[1:], ("dgamma", "dbeta", "dshift")):
            within(t, *want[k], k)


@pytest.mark.parametrize("xl", (0, 1))
@pytest.mark.parametrize("yl", (0, 1))
@pytest.mark.parametrize("xt", (0, 1))
@pytest.mark.parametrize("yt", (0, 1))
def test_norm(xt, yt, xl, yl):
    """All activations, each a copy of the code; on the largest ones in turn."""
    cases = [c for c in P.NORM if c[5:] == (xt, yt, xl, yl)]
    assert cases
    for i, (N, C, H, W, *rest) in enumerate(cases):
        norm((N, C, H, W, *rest), R.ACTS if N * C * H * W < 4 << 20 else R.ACTS[i % 5:][:1])
