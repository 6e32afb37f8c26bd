"""A UNet level from the library's operators, as they are used together.

`ResBlock` is inference: group norms feed the quantized convolutions, the time
embedding enters the second norm, and the 1x1 shortcut adds the convolution's
NCHW output to the channels-last stream:

    shift = linear(linear(t, We1, silu), We2)
    h     = conv1(norm1(x, silu))                  channels last -> NCHW
    h     = conv2(norm2(h + shift, silu))          NCHW -> NCHW
    out   = linear(x, Ws) + bias + h               channels last + NCHW -> channels last

`FeedForward` is the token-wise half, for training too: it keeps what its
backward needs and returns every gradient.

    out = x + linear(linear(norm(x), W1, gelu), W2)

Plans, weights, workspaces and outputs are made once; a call only launches.
"""
from __future__ import annotations

import torch

from .binding import Plan, wq8_conv_forward, wq8_weights_prepare
from .ops import (LinearPlan, NormPlan, wq8_linear_backward, wq8_linear_forward, wq8_norm_backward,
                  wq8_norm_forward)


class ResBlock:
    """x [N][H][W][Cin] -> [N][H][W][Cout], and the time embedding t [N][Ct].

    weights: conv1 [Cout][Cin][3][3], conv2 [Cout][Cout][3][3] (f32), norm1 and
    norm2 (gamma, beta) pairs, temb1 [E][Ct] and temb2 [Cout][E], shortcut
    [Cout][Cin] (dtype), and biases temb1_b, temb2_b, shortcut_b (f32).
    scales: s_B and s_G of the convolutions (None: 1)."""

    def __init__(self, weights, N, Cin, Cout, H, W, m=6, group=32, groups=32, s_B=None, s_G=None,
                 dtype=torch.float32, device="cuda"):
        self.w = weights
        E, Ct = weights["temb1"].shape
        f32 = torch.float32
        self.conv1 = Plan(m, N, Cin, Cout, H, W, 1, group, s_B=s_B, s_G=s_G, x_dtype=dtype)
        self.conv2 = Plan(m, N, Cout, Cout, H, W, 1, group, s_B=s_B, s_G=s_G, x_dtype=dtype)
        self.q1 = wq8_weights_prepare(self.conv1, weights["conv1"])
        self.q2 = wq8_weights_prepare(self.conv2, weights["conv2"])
        self.norm1 = NormPlan(N, Cin, H, W, groups, act="silu", x_dtype=dtype, x_layout="nhwc", y_layout="nchw")
        self.norm2 = NormPlan(N, Cout, H, W, groups, act="silu", x_dtype=dtype, x_layout="nchw")
        self.temb1 = LinearPlan(N, Ct, E, act="silu", x_dtype=dtype)
        self.temb2 = LinearPlan(N, E, Cout, x_dtype=dtype, y_dtype=f32)  # the norm's shift is f32
        self.shortcut = LinearPlan(N * H * W, Cin, Cout, x_dtype=dtype, r_layout="nchw", pixels=H * W)
        plans = (self.conv1, self.conv2, self.norm1, self.norm2, self.temb1, self.temb2, self.shortcut)
        # one stream runs them in turn: one workspace serves all
        self.ws = torch.empty(max(p.workspace_bytes for p in plans), dtype=torch.uint8, device=device)
        self.a1, self.a2 = self.norm1.empty_output(device), self.norm2.empty_output(device)
        self.h1, self.h2 = self.conv1.empty_output(device), self.conv2.empty_output(device)
        self.e1, self.shift = self.temb1.empty_output(device), self.temb2.empty_output(device)
        self.out = self.shortcut.empty_output(device)
        self.shape = (N, H, W, Cout)

    def __call__(self, x, t):
        w, ws = self.w, self.ws
        wq8_linear_forward(self.temb1, t, w["temb1"], w["temb1_b"], y=self.e1, workspace=ws)
        wq8_linear_forward(self.temb2, self.e1, w["temb2"], w["temb2_b"], y=self.shift, workspace=ws)
        wq8_norm_forward(self.norm1, x, *w["norm1"], y=self.a1, workspace=ws)
        wq8_conv_forward(self.conv1, self.a1, *self.q1, y=self.h1, workspace=ws)
        wq8_norm_forward(self.norm2, self.h1, *w["norm2"], shift=self.shift, y=self.a2, workspace=ws)
        wq8_conv_forward(self.conv2, self.a2, *self.q2, y=self.h2, workspace=ws)
        wq8_linear_forward(self.shortcut, x.view(self.shortcut.x_shape), w["shortcut"], w["shortcut_b"],
                           self.h2.view(self.shortcut.r_shape), y=self.out, workspace=ws)
        return self.out.view(self.shape)


class FeedForward:
    """x [N][H][W][C] -> x + linear(gelu(linear(norm(x)))), with its backward.

    weights: norm (gamma, beta), w1 [D][C], w2 [C][D] (dtype), b1, b2 (f32);
    they may be parameters, `backward` returns their gradients."""

    def __init__(self, weights, N, C, H, W, groups=32, dtype=torch.bfloat16, device="cuda"):
        self.w = weights
        D, rows = weights["w1"].shape[0], N * H * W
        self.norm = NormPlan(N, C, H, W, groups, x_dtype=dtype)
        self.up = LinearPlan(rows, C, D, act="gelu", x_dtype=dtype)
        self.down = LinearPlan(rows, D, C, x_dtype=dtype)
        plans = (self.norm, self.up, self.down)
        self.ws = torch.empty(max(max(p.workspace_bytes, p.backward_workspace_bytes) for p in plans), dtype=torch.uint8,
                              device=device)
        self.a, self.u, self.z = self.norm.empty_output(device), self.up.empty_output(device), self.up.empty_z(device)
        self.mean, self.rstd = self.norm.empty_stats(device)
        self.out = self.down.empty_output(device)
        self.da, self.du, self.dx = (torch.empty_like(t) for t in (self.a, self.u, self.a))

    def __call__(self, x):
        if x.requires_grad and torch.is_grad_enabled():
            raise ValueError("x requires a gradient, and no graph is recorded here: `backward` returns it")
        with torch.no_grad():
            return self._forward(x)

    def _forward(self, x):
        w, ws, rows = self.w, self.ws, self.up.x_shape
        self.x = x
        wq8_norm_forward(self.norm, x, *w["norm"], y=self.a, mean=self.mean, rstd=self.rstd, workspace=ws)
        wq8_linear_forward(self.up, self.a.view(rows), w["w1"], w["b1"], y=self.u, z=self.z, workspace=ws)
        wq8_linear_forward(self.down, self.u, w["w2"], w["b2"], x.view(rows), y=self.out, workspace=ws)
        return self.out.view(x.shape)

    @torch.no_grad()
    def backward(self, dout):
        """{name: gradient} of x and of every weight, for the last call."""
        w, ws, rows = self.w, self.ws, self.up.x_shape
        d = dout.view(rows)
        _, dw2, db2 = wq8_linear_backward(self.down, d, self.u, w["w2"], dx=self.du, want_dbias=True, workspace=ws)
        _, dw1, db1 = wq8_linear_backward(self.up, self.du, self.a.view(rows), w["w1"], z=self.z, dx=self.da.view(rows),
                                          want_dbias=True, workspace=ws)
        _, dgamma, dbeta, _ = wq8_norm_backward(self.norm, self.da, self.x, self.mean, self.rstd, *w["norm"], dx=self.dx,
                                                workspace=ws)
        return {"x": self.dx + dout, "gamma": dgamma, "beta": dbeta, "w1": dw1, "b1": db1, "w2": dw2, "b2": db2}
