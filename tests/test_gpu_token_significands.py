"""The two quotients of a row's codes, 127 / a and a / 127, are formed from an
approximate reciprocal and what it leaves: correctly rounded for every significand."""
import pytest
import torch

import quantized_convolution_amd as q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("exponent", [-90, -1, 0, 7, 99])
def test_every_significand(exponent):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    part = 1 << 20
    g = torch.Generator(device="cuda").manual_seed(exponent + 200)
    p = q.QuantPlan(part, 8)
    for at in range(0, 1 << 23, part):
        bits = (torch.arange(at, at + part, device="cuda", dtype=torch.int32) | ((exponent + 127) << 23))
        a = bits.view(torch.float32)
        x = (2 * torch.rand(part, 8, generator=g, device="cuda") - 1) * a[:, None]
        x[:, 3] = a
        most = torch.full_like(a, 127.0)
        f = most / a  # divisions of tensors, each correctly rounded
        # the halves between two codes, as near as fp32 comes: a quotient that is off moves some of them
        k = torch.randint(0, 126, (part, 3), generator=g, device="cuda") + 0.5
        x[:, 4:7] = k / f[:, None]
        codes, scales = q.wq8_quant_pack(p, x)
        assert torch.equal(scales, a / most)
        assert torch.equal(codes[:, :8].float(), torch.round(x * f[:, None]))
