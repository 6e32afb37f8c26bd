"""Every kernel instance that the plans choose (plan_cases.py), on the GPU: the
group norm against its definition in 64 bits."""
import pytest
import torch

import ops_reference as R
import plan_cases as P
import quantized_convolution_amd as q

pytestmark = pytest.mark.gpu
TYPES = (torch.float32, torch.bfloat16)
LAYOUTS = ("nhwc", "nchw")


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
