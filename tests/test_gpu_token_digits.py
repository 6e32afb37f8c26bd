"""The digits of dz in the backward of the product of codes: 32 bits where nothing
else is asked for, so that a loud token or channel takes no bits from the others,
and 16 with round_dz, in every tile."""
import pytest
import token_plan_cases as P
import token_reference as R
import torch

import quantized_convolution_amd as q

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.load()


def check(got, pair, what):
    want, bound = pair
    bad = ~((got.double() - want).abs() <= bound)
    assert got.shape == want.shape and not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()}"


def operands(seed, rows, Cin, Cout, quiet=None):
    """quiet: a token and a channel whose codes are mostly 0."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, w = r(rows, Cin), r(Cout, Cin) / Cin ** 0.5
    if quiet is not None:
        x[quiet[0], ::2] *= 1e-4
        w[quiet[1], 1::2] *= 1e-4
    return q.wq8_quant_pack(q.QuantPlan(rows, Cin), x) + q.wq8_quant_pack(q.QuantPlan(Cout, Cin), w), r


@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
@pytest.mark.parametrize("loud", [1e3, 1e5])
@pytest.mark.parametrize("rows,Cin,Cout", [(300, 70, 40), (2048, 256, 512), (1001, 333, 515)])
def test_a_loud_token_and_a_loud_channel(rows, Cin, Cout, loud, act):
    """bf16 gradients are as near as fp32 ones are, but for their own rounding."""
    print("[case] loud", rows, Cin, Cout, loud, act, flush=True)
    token, channel = rows // 3, Cout // 2
    (xq, sx, wq, sw), r = operands(rows + Cin, rows, Cin, Cout, (token, channel))
    dy = r(rows, Cout)
    dy[token] *= loud
    dy[:, channel] *= loud
    dy, z = dy.to(BF), r(rows, Cout).to(BF)
    kw = {} if act == "none" else dict(z=z)
    dx, dw, _ = q.wq8_q8linear_backward(q.Q8LinearPlan(rows, Cin, Cout, act, x_dtype=BF), dy, xq, sx, wq, sw, **kw)
    want = R.backward(dy, xq, sx, wq, sw, Cin, F32, act, z)
    for name, got in (("dx", dx), ("dw", dw)):
        v, bound = want[name]
        check(got, (v, bound + R.rounding(v, BF)), name)
    if act != "gelu":  # whose slope is off by 3e-7 at each value, loud ones too
        quiet = (xq[token, :Cin] == 0).nonzero()[:, 0]
        assert len(quiet) >= Cin // 2
        rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
        others = torch.arange(Cout, device="cuda") != channel
        v = want["dw"][0][others][:, quiet]
        # half a step of bf16 at most, and 2^-32 loud (4 deviations) of each of some thousand values
        assert rel(dw[others][:, quiet], v) <= R.BF16
        quiet = (wq[channel, :Cin] == 0).nonzero()[:, 0]
        others = torch.arange(rows, device="cuda") != token
        v = want["dx"][0][others][:, quiet]
        assert rel(dx[others][:, quiet], v) <= R.BF16


@pytest.mark.parametrize("kept", ["codes", "values"])
@pytest.mark.parametrize("rows,Cin,Cout", P.BACKWARD["bf16"])
def test_rounded_dz(rows, Cin, Cout, kept):
    print("[case] rounded dz", rows, Cin, Cout, kept, flush=True)
    (xq, sx, wq, sw), r = operands(rows + Cout, rows, Cin, Cout)
    z, dy = r(rows, Cout), r(rows, Cout).to(BF)
    dy[rows // 2] = 0
    p = q.Q8LinearPlan(rows, Cin, Cout, "gelu", x_dtype=BF, round_dz=True)
    if kept == "codes":
        zq, sz = q.wq8_quant_pack(q.QuantPlan(rows, Cout, group=32), z)
        kw, zz = dict(zq=zq, sz=sz), zq[:, :Cout].float() * sz.repeat_interleave(32, 1)[:, :Cout]
    else:
        zz = z.to(BF)
        kw = dict(z=zz)
    ws = p.empty_backward_workspace()
    ws.fill_(0x5A)
    dx, dw, db = q.wq8_q8linear_backward(p, dy, xq, sx, wq, sw, **kw, want_dbias=True, workspace=ws)
    want = R.backward(dy, xq, sx, wq, sw, Cin, BF, "gelu", zz)
    check(dx, want["dx"], "dx")
    check(dw, want["dw"], "dw")
    check(db, want["dbias"], "dbias")
    # nothing is taken from the caller who does not ask for it
    full = q.wq8_q8linear_backward(q.Q8LinearPlan(rows, Cin, Cout, "gelu", x_dtype=BF), dy, xq, sx, wq, sw, **kw, want_dbias=True)
    f32 = R.backward(dy, xq, sx, wq, sw, Cin, F32, "gelu", zz)
    for name, got in zip(("dx", "dw"), full):
        check(got, (f32[name][0], f32[name][1] + R.rounding(f32[name][0], BF)), name)
    assert torch.equal(full[2], db)


@pytest.mark.parametrize("y_dtype", [F32, BF])
def test_rounded_dz_of_borders(y_dtype):
    """An infinity or a NaN stays in its row of dx and its column's row of dw, tiny gradients are no zeros."""
    g = torch.Generator(device="cuda").manual_seed(5)
    (xq, sx, wq, sw), _ = operands(6, 140, 70, 40)
    dy = torch.randn(140, 40, generator=g, device="cuda").to(y_dtype)
    clean = dy.clone()
    dy[3, 7], dy[130, 9], clean[3, 7], clean[130, 9] = float("inf"), float("nan"), 0, 0
    p = q.Q8LinearPlan(140, 70, 40, x_dtype=BF, y_dtype=y_dtype, round_dz=True)
    dx, dw, _ = q.wq8_q8linear_backward(p, dy, xq, sx, wq, sw)
    want = R.backward(clean, xq, sx, wq, sw, 70, BF)
    rows, cols = torch.ones(140, dtype=torch.bool, device="cuda"), torch.ones(40, dtype=torch.bool, device="cuda")
    rows[[3, 130]], cols[[7, 9]] = False, False
    assert bool(torch.isnan(dx[~rows]).all()) and bool(torch.isnan(dw[~cols]).all())
    check(dx[rows], tuple(t[rows] for t in want["dx"]), "dx")
    check(dw[cols], tuple(t[cols] for t in want["dw"]), "dw")
    small = clean * 2.0 ** -110
    dx, dw, _ = q.wq8_q8linear_backward(p, small, xq, sx, wq, sw)
    want = R.backward(small, xq, sx, wq, sw, 70, BF)
    check(dx, want["dx"], "small dx")
    check(dw, want["dw"], "small dw")


@pytest.mark.parametrize("round_dz", [False, True])
def test_the_stated_bounds(round_dz):
    """dz sw itself, as products with a single code of 1 give it: off by half a unit of the fixed point (which is more
    than a half of 2^-15 or 2^-31 of the largest), and with four digits by what the sum leaves of the last one."""
    n, dtype = 128, BF if round_dz else F32
    unit = 1 / 32512 if round_dz else 1 / 2130706432
    eye = torch.eye(n, dtype=torch.int8, device="cuda")
    one = torch.ones(n, device="cuda")
    g = torch.Generator().manual_seed(1)
    k = torch.randint(0, 100 if round_dz else 1 << 20, (n, n), generator=g).double()
    k[:, 1] = 0
    dy = ((k + 0.4999) * unit).float()
    dy[:, 0] = 1
    p = q.Q8LinearPlan(n, n, n, x_dtype=dtype, y_dtype=F32, round_dz=round_dz)
    dx = q.wq8_q8linear_backward(p, dy.cuda(), eye, one, eye, one)[0].cpu().double()
    want = dy.double()
    left = 0.0 if round_dz else 2.0 ** -17 / 127
    bound = unit / 2 + left + 3 * R.U * want + R.rounding(dx, dtype)
    assert bool(((dx - want).abs() <= bound).all())
    assert bool(((dx - want)[:, 1].abs() > (2.0 ** -16 if round_dz else 2.0 ** -32)).all())
