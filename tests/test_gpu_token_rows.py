"""The norm's backward at the most rows that a plan takes, where rows count up to 2^31."""
import pytest
import torch

import quantized_convolution_amd as q

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.load()


def test_the_last_rows_of_two_to_the_31():
    """Every row of dx is written and counts in dgamma, those of the last block too: 2^31 - 1025 rows of 8 columns."""
    rows, C = (1 << 31) - 1025, 8
    need = 90 << 30  # h, which is dy too, and dx have 16 bytes a row, rstd 4: 77e9
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip("needs 90 GiB of GPU memory")
    print("[case] rows", rows, C, flush=True)
    p = q.RmsPlan(rows, C, x_dtype=BF)
    h, rstd = torch.ones(rows, C, dtype=BF, device="cuda"), torch.ones(rows, device="cuda")
    dx = torch.full((rows, C), 77.0, dtype=BF, device="cuda")
    # every value 1: n = t = 1, the mean of t n is 1, dx = 0; but for four rows of the last block and one of the first
    at = [0, rows - (1 << 20), rows - 7, rows - 2, rows - 1]
    for i, r in enumerate(at):
        h[r] = torch.arange(C, device="cuda") - 2.0 * i
    _, dgamma = q.wq8_rms_backward(p, h, h, rstd, dx=dx, dgamma=torch.empty(C, device="cuda"))
    want, part = torch.zeros(C, dtype=torch.float64), 1 << 26
    for r in at:
        v = h[r].cpu().double()
        mean = (v * v).mean()
        got = dx[r].cpu().double()
        assert bool(((got - v * (1 - mean)).abs() <= 2.0 ** -8 * got.abs()).all()), r
        want += v * v - 1
        dx[r] = 0
    for r in range(0, rows, part):
        assert not bool(dx[r:r + part].any()), r
    # sums of 2^31 ones in parts, each rounded to 24 bits some 40 times
    assert bool(((dgamma.cpu().double() - want - rows).abs() <= 64 * 2.0 ** -24 * rows).all())
    del h, dx, rstd, p
    torch.cuda.empty_cache()
