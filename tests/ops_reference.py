"""Group norm and matrix product in 64 bits, with bounds of what fp32 arithmetic
may be off by, for the GPU tests.

Bounds are worst cases of rounding to 24 bits (unit roundoff U): a sum of n
values held in fp32, joined from parts of at most 128 terms in sequence and
some tens of joins, is off by at most SUM U times the sum of magnitudes."""
import math

import torch

U = 2.0 ** -24
SUM = 256  # roundings between any value and its sum: 128 in a thread, joins, spare
BF16 = 2.0 ** -8  # half a unit in the last place of 8 significant bits, relative

# |act(a) - act(b)| <= LIP |a - b|, and the same for the slope; both sit below
# 1.13 for gelu and its tanh form, 1.10 for silu
LIP = 1.2
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z.clone()


def slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def act_error(z, name):
    """Of one evaluation: the exponential's argument is off by a few U of
    itself, and gelu's erf by 1.5e-7."""
    if name in ("none", "relu"):
        return torch.zeros_like(z)
    return 1.5e-7 * z.abs() + 8 * U * (z.abs() + 1)


def slope_error(z, name):
    if name in ("none", "relu"):
        return torch.zeros_like(z)
    return 3e-7 * (1 + z.abs()) + 16 * U * (z.abs() + 1)


def rounding(v, dtype):
    return v.abs() * (BF16 if dtype == torch.bfloat16 else U) + 1e-38


def nhwc(t, layout):
    return t if layout == "nhwc" else t.permute(0, 2, 3, 1)


class Norm:
    """One case's definition in 64 bits on NHWC views: x [N,H,W,C]."""

    def __init__(self, x, groups, eps, name, shift=None, gamma=None, beta=None):
        N, H, W, C = x.shape
        self.name, self.groups, self.shape = name, groups, x.shape
        one = torch.ones(C, dtype=torch.float64)
        self.gamma = one if gamma is None else gamma.double()
        self.beta = 0 * one if beta is None else beta.double()
        self.v = x.double() + (0 if shift is None else shift.double()[:, None, None, :])
        self.shift_error = 0 if shift is None else U * self.v.abs()
        self.mean = self.group_mean(self.v)
        d = self.v - self.spread(self.mean)
        self.rstd = 1 / torch.sqrt(self.group_mean(d * d) + eps)
        self.h = d * self.spread(self.rstd)
        self.z = self.h * self.gamma + self.beta
        self.y = act(self.z, name)

    def group_mean(self, t):
        """[N,H,W,C] -> [N,groups]"""
        N, H, W, C = self.shape
        return t.reshape(N, H * W, self.groups, C // self.groups).mean(dim=(1, 3))

    def spread(self, s):
        """[N,groups] -> [N,1,1,C]"""
        return s.repeat_interleave(self.shape[3] // self.groups, dim=1)[:, None, None, :]

    def h_error(self, mean_error, rstd_error):
        """mean_error absolute, rstd_error relative, both [N,1,1,C] or numbers."""
        return self.spread(self.rstd) * (mean_error + 2 * U * self.v.abs() + self.shift_error) + (rstd_error + 4 * U) * self.h.abs()

    def forward_errors(self, dtype):
        """Bounds of mean, rstd (relative) and y."""
        em = SUM * U * self.group_mean(self.v.abs()) + U * self.mean.abs()
        # the squared deviations: each off by its deviation's error, then summed
        dev = self.spread(em) + 2 * U * self.v.abs() + self.shift_error
        d = (self.v - self.spread(self.mean)).abs()
        er = 0.5 * self.rstd ** 2 * self.group_mean(2 * d * dev + dev ** 2) + SUM * U
        ez = self.gamma.abs() * self.h_error(self.spread(em), self.spread(er)) + 2 * U * (self.z.abs() + self.beta.abs())
        ey = LIP * ez + act_error(self.z, self.name)
        return em, er, ey + rounding(self.y, dtype)

    def backward(self, dy, dtype):
        """{name: (value, bound)}, for mean and rstd given to fp32."""
        N, H, W, C = self.shape
        P = H * W
        sp = self.spread
        dz = dy.double() * slope(self.z, self.name)
        t = self.gamma * dz
        m1, m2 = self.group_mean(t), self.group_mean(t * self.h)
        dx = sp(self.rstd) * (t - sp(m1) - self.h * sp(m2))
        eh = self.h_error(sp(U * self.mean.abs()), U)
        ez = self.gamma.abs() * eh + 2 * U * (self.z.abs() + self.beta.abs())
        edz = dy.double().abs() * (LIP * ez + slope_error(self.z, self.name)) + 2 * U * dz.abs()
        et = self.gamma.abs() * edz + U * t.abs()
        em1 = self.group_mean(et) + SUM * U * self.group_mean(t.abs())
        eth = t.abs() * eh + self.h.abs() * et
        em2 = self.group_mean(eth) + SUM * U * self.group_mean((t * self.h).abs())
        edx = sp(self.rstd) * (et + sp(em1) + self.h.abs() * sp(em2) + eh * sp(m2).abs()
                               + 6 * U * (t.abs() + sp(m1).abs() + (self.h * sp(m2)).abs())) + 2 * U * dx.abs()
        S1, S3 = dz.sum((1, 2)), self.h.sum((1, 2))
        eS1 = edz.sum((1, 2)) + SUM * U * dz.abs().sum((1, 2))
        eS3 = eh.sum((1, 2)) + SUM * U * self.h.abs().sum((1, 2))
        r, a1, a2 = (sp(q)[:, 0, 0] for q in (self.rstd, m1, m2))
        e1, e2 = (sp(q)[:, 0, 0] for q in (em1, em2))
        eshift = r * (self.gamma.abs() * eS1 + P * e1 + S3.abs() * e2 + a2.abs() * eS3
                      + 6 * U * ((self.gamma * S1).abs() + P * a1.abs() + (a2 * S3).abs()))
        eg = (edz * self.h.abs() + dz.abs() * eh).sum((0, 1, 2)) + SUM * U * (dz * self.h).abs().sum((0, 1, 2))
        eb = edz.sum((0, 1, 2)) + SUM * U * dz.abs().sum((0, 1, 2))
        return {"dx": (dx, edx + rounding(dx, dtype)), "dgamma": ((dz * self.h).sum((0, 1, 2)), eg),
                "dbeta": (dz.sum((0, 1, 2)), eb), "dshift": (dx.sum((1, 2)), eshift)}


def product(a, b, extra=0.0):
    """a [M,K] times b [N,K]^T in 64 bits, and the bound of fp32 sums of
    products in any order; `extra`: relative error of a's entries."""
    a, b = a.double(), b.double()
    mags = a.abs() @ b.abs().T
    return a @ b.T, (2 * (a.shape[1] + 8) * U + extra) * mags


def linear_forward(x, w, bias, residual, name, dtype):
    """((y, bound), (z, bound)); residual [M,N] or None."""
    z, ez = product(x, w)
    if bias is not None:
        z = z + bias.double()
        ez = ez + U * (z.abs() + bias.double().abs())
    y = act(z, name)
    ey = LIP * ez + act_error(z, name)
    if residual is not None:
        y = y + residual.double()
        ey = ey + U * y.abs()
    return (y, ey + rounding(y, dtype)), (z, ez + rounding(z, dtype))


def linear_backward(dy, x, w, z, name, x_dtype, rounds):
    """{name: (value, bound)}; rounds: dz is rounded to bf16 on its way into the products."""
    dz = dy.double()
    edz = torch.zeros_like(dz)
    if name != "none":
        edz = dz.abs() * slope_error(z.double(), name) + 2 * U * (dz * slope(z.double(), name)).abs()
        dz = dz * slope(z.double(), name)
    ed = edz + (BF16 * dz.abs() if rounds else 0)
    dx, ex = product(dz, w.T)
    dw, ew = product(dz.T, x.T)
    ex = ex + ed @ w.double().abs() + rounding(dx, x_dtype)
    ew = ew + ed.T @ x.double().abs() + rounding(dw, x_dtype)
    return {"dx": (dx, 1.01 * ex), "dw": (dw, 1.01 * ew),
            "dbias": (dz.sum(0), edz.sum(0) + 2 * (SUM + 64) * U * dz.abs().sum(0))}


def check(got, want, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = (got - want).abs()
    worst = (off - bound).max().item() if off.numel() else 0.0
    assert not torch.isnan(off).any(), f"{what}: NaN"
    assert worst <= 0, f"{what}: off by {off.max().item():.3e}, {worst:.3e} over its bound"
