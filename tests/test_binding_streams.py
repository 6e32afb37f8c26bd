"""What the convolution's binding allocates for a call on another stream is that
stream's: torch's allocator hands a freed block out again in the order of the
stream that it belongs to."""
import contextlib

import pytest
import torch

from quantized_convolution_amd import binding as B


def calls():
    p = B.Plan(4, 1, 32, 16, 8, 8, 1, 32)
    f32, i8 = torch.float32, torch.int8
    x, w = torch.zeros(p.x_shape), torch.zeros(16, 32, 3, 3)
    Uq, sU = torch.zeros(p.uq_shape, dtype=i8), torch.zeros(p.su_shape)
    Vq, sV, M = torch.zeros(p.vq_shape, dtype=i8), torch.zeros(p.sv_shape), torch.zeros(p.m_shape)
    wq, sw, xq, sx = (torch.zeros(s, dtype=t) for s, t in zip(B._direct_shapes(p), (i8, f32, i8, f32)))
    return [("wq8_weights_prepare", (w,)), ("wq8_conv_forward", (x, Uq, sU)), ("wq8_stage1", (x,)),
            ("wq8_stage2", (Vq, sV, Uq, sU)), ("wq8_stage2_i32", (Vq, Uq)), ("wq8_stage3", (M,)),
            ("wq8_stage23", (Vq, sV, Uq, sU)), ("wq8_direct_weights_prepare", (w,)), ("wq8_direct_quantize_x", (x,)),
            ("wq8_direct_conv", (xq, sx, wq, sw)), ("wq8_direct_forward", (x, wq, sw))], p


@pytest.mark.parametrize("which", range(11))
def test_allocations_belong_to_the_stream(monkeypatch, which):
    cases, plan = calls()
    name, args = cases[which]
    made, inside = [], []
    real = torch.empty

    def empty(*a, **kw):
        made.append(list(inside))
        return real(*a, **{**kw, "device": "cpu"})

    @contextlib.contextmanager
    def stream(s):
        inside.append(s)
        yield
        inside.pop()

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(B._Bufs, "call", lambda self, fn, *a, stream=None: None)
    getattr(B, name)(plan, *args, stream="another stream")
    assert made and all(m == ["another stream"] for m in made) and not inside
    made.clear()
    getattr(B, name)(plan, *args)
    assert made and not any(made)
