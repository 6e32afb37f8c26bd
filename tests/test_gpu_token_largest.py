"""The operators on 8-bit codes at the most rows and columns that they are documented
for: places that count past 31 bits, launches of several rows of blocks, and
strides of 2^24 bytes between the columns of a transposed operand."""
import pytest
import token_reference as R
import torch

import quantized_convolution_amd as q

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def room():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 160 GiB of GPU memory")
    yield
    torch.cuda.empty_cache()


def check(got, pair, what):
    want, bound = pair
    bad = ~((got.double() - want).abs() <= bound)
    assert got.shape == want.shape and not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()}"


PERIOD = 1 << 12  # rows of a pattern that is repeated


def repeated(t, rows):
    return t.repeat(-(-rows // len(t)), *[1] * (t.dim() - 1))[:rows].contiguous()


def repeats(t, small):
    """Whether t's rows are those of `small` over and over."""
    whole = len(t) // len(small) * len(small)
    parts = t[:whole].view(-1, *small.shape)
    step = max(1, (1 << 28) // small.numel())
    return all(bool((parts[i:i + step] == small).all()) for i in range(0, len(parts), step)) and torch.equal(t[whole:], small[:len(t) - whole])


@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_packing_past_31_bits(group):
    """2^34 values and some: 2^31 threads."""
    rows, C = (1 << 27) + 77, 128
    print("[case] pack", rows, C, group, flush=True)
    g = torch.Generator(device="cuda").manual_seed(group)
    small = torch.randn(PERIOD, C, generator=g, device="cuda").to(BF)
    want = q.wq8_quant_pack(q.QuantPlan(PERIOD, C, group, x_dtype=BF), small)
    values = q.wq8_quant_unpack(q.QuantPlan(PERIOD, C, group, x_dtype=BF), *want)
    p, x = q.QuantPlan(rows, C, group, x_dtype=BF), repeated(small, rows)
    codes, scales = q.wq8_quant_pack(p, x)
    assert repeats(codes, want[0]) and repeats(scales, want[1])
    x.fill_(float("nan"))
    assert repeats(q.wq8_quant_unpack(p, codes, scales, x=x), values)


def test_norm_of_many_rows():
    rows, C = (1 << 27) + 77, 72
    print("[case] norm", rows, C, flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    small, gm = torch.randn(PERIOD, C, generator=g, device="cuda").to(BF), 1 + 0.1 * torch.randn(C, generator=g, device="cuda")
    want = q.wq8_rms_forward(q.RmsPlan(PERIOD, C, x_dtype=BF), small, gm, small, want_codes=True, want_rstd=True)
    x = repeated(small, rows)
    got = q.wq8_rms_forward(q.RmsPlan(rows, C, x_dtype=BF), x, gm, x, h=x, want_codes=True, want_rstd=True)
    assert all(repeats(a, b) for a, b in zip(got, want))


def test_many_rows_of_few_and_of_many_columns():
    """Rows that are read twice, more of them than one row of blocks has."""
    for rows, C in (((1 << 22) + 3, 5), ((1 << 21) + 5, 7)):
        print("[case] norm", rows, C, flush=True)
        g = torch.Generator(device="cuda").manual_seed(C)
        small, dy = (torch.randn(PERIOD, C, generator=g, device="cuda") for _ in range(2))
        p, p1 = q.RmsPlan(rows, C), q.RmsPlan(PERIOD, C)
        want = q.wq8_rms_forward(p1, small, want_codes=True, want_rstd=True)
        x = repeated(small, rows)
        got = q.wq8_rms_forward(p, x, want_codes=True, want_rstd=True)
        assert all(repeats(a, b) for a, b in zip(got, want))
        dx, dg = q.wq8_rms_backward(p, repeated(dy, rows), x, got[4], dgamma=torch.empty(C, device="cuda"))
        assert repeats(dx, q.wq8_rms_backward(p1, dy, small, want[4])[0])
        terms = repeated(dy, rows).double() * x.double() * got[4].double()[:, None]
        # parts of some 16384 rows in turn, and their joins
        check(dg, (terms.sum(0), (rows // 256 + 256) * R.U * terms.abs().sum(0)), "dgamma")


@pytest.mark.parametrize("C", [(1 << 20) - 1, (1 << 20) - 8])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_norm_of_the_most_columns(C, dtype):
    print("[case] norm", C, dtype, flush=True)
    g = torch.Generator().manual_seed(C)
    x, dy = (torch.randn(3, C, generator=g).to(dtype) for _ in range(2))
    gm = 1 + 0.1 * torch.randn(C, generator=g)
    p = q.RmsPlan(3, C, x_dtype=dtype)
    y, _, codes, scales, rstd = q.wq8_rms_forward(p, x.cuda(), gm.cuda(), want_codes=True, want_rstd=True)
    ref = R.Rms(x, 1e-6, gm)
    # a thread has 1024 columns here, in parts of 8, where the reference's bounds count on 128
    more = 1024 * R.U
    f = ref.forward(dtype)
    check(rstd.cpu(), (f["rstd"][0], f["rstd"][1] + more * f["rstd"][0]), "rstd")
    check(y.cpu(), (f["y"][0], f["y"][1] + more * f["y"][0].abs()), "y")
    t = R.codes_of(x.float().numpy() * gm.numpy())
    assert torch.equal(codes.cpu(), t[0])
    s = ref.scales(t[1])
    check(scales.cpu(), (s[0], s[1] + more * s[0]), "scales")
    dx, dg = q.wq8_rms_backward(p, dy.cuda(), x.cuda(), rstd, gm.cuda())
    want = ref.backward(dy, rstd.cpu(), None, dtype)
    n = x.double() * rstd.cpu().double()[:, None]
    mean = (gm.double() * dy.double() * n).abs().mean(1, keepdim=True)
    check(dx.cpu(), (want["dx"][0], want["dx"][1] + more * rstd.cpu().double()[:, None] * n.abs() * mean), "dx")
    check(dg.cpu(), want["dgamma"], "dgamma")
    pack = q.QuantPlan(3, C, x_dtype=dtype)
    codes, scales = q.wq8_quant_pack(pack, x.cuda())
    t = R.codes_of(x.float().numpy())
    assert torch.equal(codes.cpu(), t[0]) and torch.equal(scales.cpu(), t[1])


@pytest.mark.parametrize("dtype,round_dz", [(F32, False), (BF, False), (BF, True)])
def test_product_of_the_most_rows(dtype, round_dz):
    """2^24 - 1 tokens: dw sums over all of them, in splits of k."""
    rows, Cin, Cout = (1 << 24) - 1, 40, 70
    print("[case] product", rows, Cin, Cout, dtype, round_dz, flush=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    xs, ws = q.wq8_quant_pack(q.QuantPlan(PERIOD, Cin), r(PERIOD, Cin)), q.wq8_quant_pack(q.QuantPlan(Cout, Cin), r(Cout, Cin))
    dys, bias = r(PERIOD, Cout).to(dtype), r(Cout)
    make = lambda n: q.Q8LinearPlan(n, Cin, Cout, "silu", x_dtype=dtype, round_dz=round_dz)  # noqa: E731
    small, p = make(PERIOD), make(rows)
    y, z, zq, sz = q.wq8_q8linear_forward(small, *xs, *ws, bias, want_z=True, want_zq=True)
    xq, sx = (repeated(t, rows) for t in xs)
    got = q.wq8_q8linear_forward(p, xq, sx, *ws, bias, want_z=True, want_zq=True)
    assert all(repeats(a, b) for a, b in zip(got, (y, z, zq, sz)))
    dy = repeated(dys, rows)
    full = q.wq8_q8linear_backward(p, dy, xq, sx, *ws, z=got[1], want_dbias=True)
    assert repeats(full[0], q.wq8_q8linear_backward(small, dys, *xs, *ws, z=z)[0])
    # a few tokens with a gradient, at both ends and where a split of k ends: all of dw is theirs
    at = torch.tensor([0, 1, 65535, 65536, rows // 2, rows - 3, rows - 2, rows - 1], device="cuda")
    few = dy[at]
    dy.zero_()
    dy[at] = few
    _, dw, db = q.wq8_q8linear_backward(p, dy, xq, sx, *ws, z=got[1], want_dx=False, want_dbias=True)
    want = R.backward(few, xq[at], sx[at], *ws, Cin, dtype, "silu", got[1][at].float())
    check(dw, want["dw"], "dw")
    check(db, want["dbias"], "dbias")
    # every token: the sum over the pattern, so many times; parts of k and of the rows are joined in fp32
    del dy
    count, more = rows // PERIOD, slice(0, rows % PERIOD)
    one, rest = (R.backward(dys[i], xs[0][i], xs[1][i], *ws, Cin, dtype, "silu", z[i].float()) for i in (slice(None), more))
    for name, v in (("dw", full[1]), ("dbias", full[2])):
        check(v, (count * one[name][0] + rest[name][0], 2 * (count * one[name][1] + rest[name][1])), name)


@pytest.mark.parametrize("rows,Cin,Cout", [(2, (1 << 20) - 1, 33), (40, (1 << 20) - 1, 33), (5, 40, (1 << 20) - 1), (300, 40, (1 << 20) - 1)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_product_of_the_most_columns(rows, Cin, Cout, dtype):
    print("[case] product", rows, Cin, Cout, dtype, flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    xq, sx = q.wq8_quant_pack(q.QuantPlan(rows, Cin), r(rows, Cin))
    wq, sw = q.wq8_quant_pack(q.QuantPlan(Cout, Cin), r(Cout, Cin))
    p, bias = q.Q8LinearPlan(rows, Cin, Cout, "relu", x_dtype=dtype), r(Cout)
    y, z, zq, sz = q.wq8_q8linear_forward(p, xq, sx, wq, sw, bias, want_z=True, want_zq=True)
    acc = xq[:, :Cin].double() @ wq[:, :Cin].double().T
    want = acc.float() * sx[:, None] * sw[None, :] + bias
    assert torch.equal(z, want.to(dtype)) and torch.equal(y, torch.relu(want).to(dtype))
    codes = q.wq8_quant_pack(q.QuantPlan(rows, Cout, group=32), want)
    assert torch.equal(zq, codes[0]) and torch.equal(sz, codes[1])
    dy = r(rows, Cout).to(dtype)
    dx, dw, db = q.wq8_q8linear_backward(p, dy, xq, sx, wq, sw, z=z, want_dbias=True)
    ref = R.backward(dy, xq, sx, wq, sw, Cin, dtype, "relu", z.float())
    check(dx, ref["dx"], "dx")
    check(dw, ref["dw"], "dw")
    check(db, ref["dbias"], "dbias")
