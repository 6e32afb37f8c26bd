"""The activations' slopes in the backward of the product of codes, value by value:
with one row dbias is dy act'(z) in fp32."""
import math

import pytest
import token_reference as R
import torch

import quantized_convolution_amd as q

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
U = R.U


@pytest.fixture(scope="module", autouse=True)
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.load()


def slopes(z, act, dtype, codes=None):
    n = z.shape[0]
    p = q.Q8LinearPlan(1, 8, n, act, x_dtype=dtype)
    a = torch.zeros(1, 128, dtype=torch.int8, device="cuda"), torch.ones(1, device="cuda"), torch.zeros(n, 128, dtype=torch.int8, device="cuda")
    kw = dict(z=z[None].cuda()) if codes is None else dict(zip(("zq", "sz"), (t.cuda() for t in codes)))
    got = q.wq8_q8linear_backward(p, torch.ones(1, n, dtype=dtype, device="cuda"), *a, torch.ones(n, device="cuda"), **kw, want_dbias=True)
    return got[2].cpu().double()


def gelu_bound(z):
    """Of a slope from Abramowitz and Stegun's 7.1.26 in fp32: what the formula itself is off by, in 64 bits, and 32
    roundings of its terms, with the exponential's argument z^2 / 2 rounded twice."""
    a = z.abs()
    t = 1 / (1 + 0.3275911 * a / math.sqrt(2))
    e = torch.exp(-a * a / 2)
    cdf = 0.5 * t * e * (0.254829592 + t * (-0.284496736 + t * (1.421413741 + t * (-1.453152027 + t * 1.061405429))))
    true = 0.5 * torch.special.erfc(a / math.sqrt(2))
    density = a * e / math.sqrt(2 * math.pi)
    return (cdf - true).abs() + (32 + 2 * z * z) * U * (cdf + density) + torch.where(z >= 0, U, 0.0) + 1e-37


@pytest.mark.parametrize("kept", ["values", "codes"])
def test_gelu_slope_in_both_tails(kept):
    """bf16 results: the negative tail is no difference of numbers near 1/2."""
    z = torch.cat([torch.linspace(-9, 9, 5761), torch.tensor([-12.0, -10.0, -1e-3, 0.0, -0.0, 1e-3, 10.0, 40.0, -40.0, 1e18, -1e18])]).to(BF)
    codes = None
    if kept == "codes":
        codes = R.codes_of(z[None, :5760].float().numpy(), 32)
        z = (codes[0][0, :5760].float() * codes[1][0].repeat_interleave(32))
    got = slopes(z, "gelu", BF, codes)
    zz = z.double()
    want, bound = R.slope(zz, "gelu"), gelu_bound(zz)
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), [(float(zz[i]), float(got[i]), float(want[i]), float(bound[i])) for i in bad.nonzero()[:5, 0]]
    # some thousandths of the slope itself, as far down as it is a normal number, but about its zero
    far = (zz < -2) & (want.abs() > 1e-30)
    assert bool(((got - want).abs()[far] <= 4e-3 * want[far].abs()).all())


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_slopes_of_borders(act, dtype):
    """A NaN stays; infinities are as the formulas give them, the same for both types."""
    z = torch.tensor([math.nan, math.inf, -math.inf, 0.0, 3e38, -3e38]).to(dtype)
    got = slopes(z, act, dtype)
    assert math.isnan(got[0])
    if act == "relu":
        assert got[1:].tolist() == [1, 0, 0, 1, 0]
    else:
        assert bool(torch.isnan(got[1:3]).all()) or got[1:3].tolist() == [1, 0]
        # at 0 the slope is the distribution function's 1/2: to 7 roundings of fp32, or to 1.5e-7
        assert abs(got[3] - 0.5) <= (7 * U * 0.5 if dtype == F32 else 1.5e-7 + U) and got[4:].tolist() == [1, 0]
    other = F32 if dtype == BF else BF
    assert torch.equal(torch.isnan(got), torch.isnan(slopes(z.to(other), act, other)))
