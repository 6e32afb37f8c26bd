"""A transformer block's feed forward from the operators on 8-bit codes, as they
are used together, for serving and for training:

    h   = x + residual;  out = h + linear(gelu(linear(rms(h), W1)), W2)

Both products run on 8-bit codes: the norm hands its own on, the inner
activations are packed. What the backward needs is kept in 8 bits (codes of both
products' inputs and of the first one's z), beside the stream h and one number a
row: 1 + 4 (1 + 1.125) = 9.5 bytes a value of the stream for an inner width of 4 C,
where bf16 activations would be 2 (1 + 4 + 4) = 18. The block also owns the buffers
that it works in for as long as it lives: in bf16 the inner activations and their
gradient (8 + 8), the stream, the output and two gradients of it (2 each), 24 bytes a
value more. One block serves layers one after the other only if their backwards
follow their calls; a block for each layer holds them for each.
"""
from __future__ import annotations

import torch

from .token_ops import (Q8LinearPlan, QuantPlan, RmsPlan, wq8_q8linear_backward, wq8_q8linear_forward, wq8_quant_pack,
                        wq8_rms_backward, wq8_rms_forward)


def _is(x, own):
    """Whether x, a tensor of own's form, is the memory of own."""
    return isinstance(x, torch.Tensor) and x.shape == own.shape and x.dtype == own.dtype and x.is_contiguous() and \
        x.data_ptr() == own.data_ptr() and x.device == own.device


class Q8FeedForward:
    """x [rows][C], a residual of its shape or None -> out [rows][C].

    weights: gamma [C] (f32), w1 [D][C], w2 [C][D] (dtype), b1 [D], b2 [C] (f32);
    they may be parameters. They are packed when the block is made and by `pack`,
    after they change; `backward` returns their gradients, those of the packed
    weights as the weights' own. Plans, workspaces and outputs are made once; a
    call only launches, and the next one writes over what it returned. train=False
    keeps nothing for a backward.

    Without a residual x itself is the stream that `backward` reads: it stays as it
    is until then. What the block has returned may be given to it again (it is
    copied, since the call, or its backward, writes over it)."""

    def __init__(self, weights, rows, C, dtype=torch.bfloat16, eps=1e-6, act="gelu", train=True, device="cuda"):
        self.w, self.train = weights, train
        D = weights["w1"].shape[0]
        self.norm = RmsPlan(rows, C, eps, x_dtype=dtype)
        self.up = Q8LinearPlan(rows, C, D, act=act, x_dtype=dtype)
        self.down = Q8LinearPlan(rows, D, C, x_dtype=dtype)
        self.inner = QuantPlan(rows, D, x_dtype=dtype)
        self.plans1, self.plans2 = QuantPlan(D, C, x_dtype=dtype), QuantPlan(C, D, x_dtype=dtype)
        self.w1, self.w2 = self.plans1.empty_codes(device), self.plans2.empty_codes(device)
        plans = (self.norm, self.up, self.down)
        need = [p.workspace_bytes for p in plans] + [p.backward_workspace_bytes for p in plans if train]
        self.ws = torch.empty(max(need), dtype=torch.uint8, device=device)
        self.a, self.rstd = self.norm.empty_codes(device), self.norm.empty_rstd(device) if train else None
        self.h, self.u, self.uq = self.norm.empty_input(device), self.up.empty_output(device), self.inner.empty_codes(device)
        self.z = self.up.empty_z_codes(device) if train and act != "none" else (None, None)
        self.out, self.stream = self.down.empty_output(device), None
        if train:
            self.du, self.da, self.dx = (torch.empty_like(t) for t in (self.u, self.h, self.h))
        self.pack()

    @torch.no_grad()
    def pack(self):
        """Packs the weights as they are now."""
        wq8_quant_pack(self.plans1, self.w["w1"], *self.w1)
        wq8_quant_pack(self.plans2, self.w["w2"], *self.w2)

    def __call__(self, x, residual=None):
        for t in (x, residual):
            if t is not None and t.requires_grad and torch.is_grad_enabled():
                raise ValueError("an input requires a gradient, and no graph is recorded here: `backward` returns it")
        with torch.no_grad():
            return self._forward(x, residual)

    def _forward(self, x, residual):
        w, ws = self.w, self.ws
        h = None if residual is None else self.h
        if self.train and h is None and (_is(x, self.out) or _is(x, self.dx)):
            x = self.h.copy_(x)
        wq8_rms_forward(self.norm, x, w["gamma"], residual, h=h, codes=self.a[0], scales=self.a[1], rstd=self.rstd, want_y=False,
                        workspace=ws)
        self.stream = x if residual is None else h
        wq8_q8linear_forward(self.up, *self.a, *self.w1, w["b1"], y=self.u, zq=self.z[0], sz=self.z[1], workspace=ws)
        wq8_quant_pack(self.inner, self.u, *self.uq)
        return wq8_q8linear_forward(self.down, *self.uq, *self.w2, w["b2"], self.stream, y=self.out, workspace=ws)

    @torch.no_grad()
    def backward(self, dout):
        """{name: gradient} for the last call; "x" is that of x and of the residual."""
        if not self.train:
            raise ValueError("made with train=False: nothing is kept for a backward")
        if self.stream is None:
            raise ValueError("nothing has been called yet that this could be the backward of")
        w, ws = self.w, self.ws
        _, dw2, db2 = wq8_q8linear_backward(self.down, dout, *self.uq, *self.w2, dx=self.du, want_dbias=True, workspace=ws)
        _, dw1, db1 = wq8_q8linear_backward(self.up, self.du, *self.a, *self.w1, zq=self.z[0], sz=self.z[1], dx=self.da,
                                            want_dbias=True, workspace=ws)
        _, dgamma = wq8_rms_backward(self.norm, self.da, self.stream, self.rstd, w["gamma"], dh=dout, dx=self.dx, workspace=ws)
        return {"x": self.dx, "gamma": dgamma, "w1": dw1, "b1": db1, "w2": dw2, "b2": db2}
