"""Infinities and NaN in z, through every kernel of the product of codes: the same
for both types, and as the activations' formulas give them."""
import math

import pytest
import torch

import quantized_convolution_amd as q

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.load()


WANT = {  # of +infinity, -infinity, NaN, 1e38 and -1e38; -infinity times a gate of 0 is a NaN
    "none": [math.inf, -math.inf, math.nan, 1e38, -1e38], "relu": [math.inf, 0.0, math.nan, 1e38, 0.0],
    "silu": [math.inf, math.nan, math.nan, 1e38, 0.0], "gelu": [math.inf, math.nan, math.nan, 1e38, 0.0],
    "gelu_tanh": [math.inf, math.nan, math.nan, 1e38, 0.0],
}


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("act", list(WANT))
@pytest.mark.parametrize("rows,Cin,Cout", [(1, 40, 45), (2, 300, 64), (5, 300, 45), (40, 300, 45), (700, 139, 649), (1024, 256, 1024),
                                           (4096, 512, 4096), (154, 6569, 5551)])
def test_bias(rows, Cin, Cout, act, dtype):
    print("[case] infinities", rows, Cin, Cout, act, dtype, flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, w = torch.randn(rows, Cin, generator=g, device="cuda"), torch.randn(Cout, Cin, generator=g, device="cuda")
    a = q.wq8_quant_pack(q.QuantPlan(rows, Cin), x) + q.wq8_quant_pack(q.QuantPlan(Cout, Cin), w)
    bias = torch.zeros(Cout, device="cuda")
    at = torch.tensor([0, 7, 13, 31, Cout - 1], device="cuda")
    bias[at] = torch.tensor([math.inf, -math.inf, math.nan, 1e38, -1e38], device="cuda")
    y = q.wq8_q8linear_forward(q.Q8LinearPlan(rows, Cin, Cout, act, x_dtype=dtype), *a, bias).float()
    want = torch.tensor(WANT[act], device="cuda").to(dtype).float().expand(rows, 5)
    got = y[:, at]
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert bool((got[ok] == want[ok]).all())
    others = torch.ones(Cout, dtype=torch.bool)
    others[at.cpu()] = False
    assert bool(torch.isfinite(y[:, others.cuda()]).all())
