"""The operators on 8-bit codes in 64 bits, with bounds of what fp32 arithmetic
may be off by, for the GPU tests.

Codes are defined to the bit (one fp32 quotient, one fp32 product, nearest even),
so they are compared as they are. Everything else has a worst case of rounding to
24 bits (unit roundoff U): a sum of n values held in fp32, joined from parts of
at most 128 terms in sequence and some tens of joins, is off by at most SUM U
times the sum of magnitudes."""
import numpy as np
import torch

from ops_reference import BF16, LIP, SUM, U, act, act_error, rounding, slope, slope_error  # noqa: F401

F32, BF = torch.float32, torch.bfloat16


def stride(columns):
    return (columns + 127) // 128 * 128


def codes_of(x, group=0):
    """(codes [rows][stride], scales) of fp32 values (numpy), to the bit."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    rows, C = x.shape
    n = group or C
    codes = np.zeros((rows, stride(C)), np.int8)
    scales = np.zeros((rows, -(-C // n)), np.float32)
    with np.errstate(all="ignore"):
        for j in range(scales.shape[1]):
            v = x[:, j * n:(j + 1) * n]
            a = np.max(np.abs(v), axis=1, initial=0.0).astype(np.float32)  # NaN where there is one
            bad = ~np.isfinite(a)
            up = np.where(a < np.float32(2.0 ** -100), np.float32(2.0 ** 64), np.float32(1))
            f = np.where((a == 0) | bad, np.float32(0), np.float32(127) / (a * up)).astype(np.float32)
            q = np.rint((v * up[:, None]).astype(np.float32) * f[:, None])
            codes[:, j * n:j * n + v.shape[1]] = np.where(bad[:, None], 0, q).astype(np.int8)
            scales[:, j] = np.where(bad, np.float32(np.nan), a / np.float32(127))
    return torch.from_numpy(codes), torch.from_numpy(scales if group else scales[:, 0].copy())


def values(codes, scales, C, group=0):
    """What codes stand for, in 64 bits."""
    v = codes[:, :C].double()
    if not group:
        return v * scales.double()[:, None]
    return v * scales.double().repeat_interleave(group, dim=1)[:, :C]


# ---------------------------------------------------------------------- norm
RSTD = 0.5 * SUM + 4  # roundings of 1 / sqrt(sum / C + eps): half of the sum's, the quotients' and the root's


class Rms:
    """h: the stream, already rounded to its type."""

    def __init__(self, h, eps, gamma=None):
        self.C = h.shape[1]
        self.h = h.double()
        self.gamma = torch.ones(self.C, dtype=torch.float64) if gamma is None else gamma.double()
        self.rstd = 1 / torch.sqrt(self.h.square().sum(1) / self.C + eps)
        self.y = self.h * self.rstd[:, None] * self.gamma

    def forward(self, dtype):
        """{name: (value, bound)}"""
        return {"rstd": (self.rstd, RSTD * U * self.rstd),
                "y": (self.y, (RSTD + 2) * U * self.y.abs() + rounding(self.y, dtype))}

    def scales(self, scale):
        """Of the codes: `scale` of those of h gamma, times rstd."""
        s = scale.double() * self.rstd
        return s, (RSTD + 1) * U * s + 1e-44

    def backward(self, dy, rstd, dh, dtype):
        """For rstd as given, in fp32."""
        r = rstd.double()[:, None]
        n, dy = self.h * r, dy.double()
        t = self.gamma * dy
        m = (t * n).sum(1, keepdim=True) / self.C
        em = (SUM + 4) * U * (t * n).abs().sum(1, keepdim=True) / self.C
        core = r * (t - n * m)
        # t and n one rounding each, their product's difference one more, then rstd
        e = r * (n.abs() * em + 3 * U * (t.abs() + (n * m).abs())) + 2 * U * core.abs()
        dx = core
        if dh is not None:
            dx = core + dh.double()
            e = e + U * dx.abs()
        dg = (dy * n).sum(0)
        return {"dx": (dx, e + rounding(dx, dtype)), "dgamma": (dg, (SUM + 4) * U * (dy * n).abs().sum(0) + 1e-38)}


# ------------------------------------------------------------------- product
def product(xq, sx, wq, sw, Cin, bias=None):
    """z in fp32 to the bit: an exact whole number, rounded, times the two scales, plus the bias."""
    acc = xq[:, :Cin].double() @ wq[:, :Cin].double().T  # below 2^53
    z = acc.float().numpy() * sx.float().numpy()[:, None]
    z = (z * sw.float().numpy()[None, :]).astype(np.float32)
    if bias is not None:
        z = z + bias.float().numpy()[None, :]
    return torch.from_numpy(z.astype(np.float32))


def forward(z, name, residual, dtype):
    """(y, bound) of z as product() has it."""
    z = z.double()
    y = act(z, name)
    e = act_error(z, name)
    if residual is not None:
        y = y + residual.double()
        e = e + U * y.abs()
    return y, e + rounding(y, dtype)


def backward(dy, xq, sx, wq, sw, Cin, dtype, name="none", z=None):
    """{name: (value, bound)}; z: the values that the backward has, exactly."""
    dz, edz = dy.double(), 0 * dy.double()
    if name != "none":
        z = z.double()
        s = slope(z, name)
        edz = dz.abs() * (slope_error(z, name) + 2 * U * (z.abs() + 1))
        dz = dz * s
        edz = edz + U * dz.abs()
    xc, wc = xq[:, :Cin].double(), wq[:, :Cin].double()
    sx, sw = sx.double(), sw.double()

    def one(u, eu, c, along):
        """u [m][k] times whole numbers c [k][n], u held to a part of its rows' largest."""
        step = 2.0 ** -16 if dtype == BF else 2.0 ** -32
        most = u.abs().amax(1, keepdim=True)
        eu = eu + step * 1.01 * most + 3 * U * u.abs()  # scale, factor and product of the fixed point
        v = u @ c
        e = eu @ c.abs() + 20 * U * (u.abs() @ c.abs())  # joins of parts of the sum, and what follows
        if dtype != BF:  # the lowest digits' bits: half of 2^-16 in units of the highest digit
            e = e + 2.0 ** -17 * 1.01 * most / 127 * (1 + 0 * v)
        return v, e + 4 * U * v.abs() + rounding(v, dtype)

    u = dz * sw
    dx = one(u, edz * sw + U * u.abs(), wc, 1)
    u = (dz * sx[:, None]).T
    dw = one(u, (edz * sx[:, None]).T + U * u.abs(), xc, 0)
    db = dz.sum(0)
    return {"dx": dx, "dw": dw, "dbias": (db, edz.sum(0) + (SUM + 4) * U * dz.abs().sum(0) + 1e-38)}
