"""Cases for the 8-bit operators of a transformer block's products: the
root-mean-square norm with the residual's addition and an output in 8 bits, the
packing of rows to 8 bits, the matrix product of 8-bit codes with scales for
each token and channel, and its backward from what was kept in 8 bits.

`listed()` gives named cases, `draw(rng)` further ones of the same ranges.
`prepare` makes a case's inputs from a seed, `run` makes one pass: with `own`
set through the framework's entry points, else in plain torch operations in
32 bits. `exact` evaluates the definitions in 64 bits, `work` counts the bytes
and operations that a pass cannot do without. What is held in 8 bits is
returned as the values it stands for.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6
Z_GROUP = 32  # columns that share a scale where a product's z is kept in 8 bits

# Cost bounds of drawn cases: the largest listed ones (values of a tensor,
# multiply-adds of one product).
MAX_VALUES = 16384 * 5120
MAX_PRODUCT = 16384 * 2560 * 10240


def _rms(op, rows, C, x_dtype, y_dtype, residual=False, q8=False, dh=False, x_stride=0, name=None):
    case = dict(op=op, rows=rows, C=C, x_dtype=x_dtype, y_dtype=y_dtype, residual=residual, q8=q8, dh=dh, x_stride=x_stride)
    return dict(case, name=name) if name else case


def _pack(rows, C, group, x_dtype, x_stride=0, name=None):
    case = dict(op="pack", rows=rows, C=C, group=group, x_dtype=x_dtype, x_stride=x_stride)
    return dict(case, name=name) if name else case


def _q8(op, rows, Cin, Cout, act, x_dtype, y_dtype, bias=True, residual="none", pixels=0, z="none", pack=False, y_stride=0,
        name=None):
    case = dict(op=op, rows=rows, Cin=Cin, Cout=Cout, act=act, x_dtype=x_dtype, y_dtype=y_dtype, bias=bias, residual=residual,
                pixels=pixels, z=z, pack=pack, y_stride=y_stride)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one token of a stream of 1280 channels, in front of an 8-bit product: latency
        _rms("rms_fwd", 1, 1280, "bf16", "bf16", residual=True, q8=True, name="rms_1x1280_bf16_q8"),
        # a wide block's tokens, the largest norm: bound by memory
        _rms("rms_fwd", 16384, 2560, "bf16", "bf16", residual=True, q8=True, name="rms_16384x2560_bf16_q8"),
        # 32 bits, odd rows that are a slice of a wider tensor, an output in 32 bits
        _rms("rms_fwd", 1001, 1285, "f32", "f32", x_stride=1288, name="rms_1001x1285_f32_strided"),
        # training at the 1280-channel layer: the stream's own gradient joins in
        _rms("rms_bwd", 8192, 1280, "bf16", "bf16", dh=True, name="rms_bwd_8192x1280_bf16"),
        # training in 32 bits at an odd width
        _rms("rms_bwd", 1001, 333, "f32", "f32", name="rms_bwd_1001x333_f32"),
        # the feed forward's inner activations between its two products: one scale a token
        _pack(8192, 5120, 0, "bf16", name="pack_8192x5120_bf16_rows"),
        # an activation kept for the backward pass in groups of 32, odd width, 32 bits
        _pack(1001, 2565, 32, "f32", name="pack_1001x2565_f32_g32"),
        # one token through a wide product, activations as they come: bound by the weights' bytes
        _q8("q8_fwd", 1, 10240, 10240, "none", "bf16", "bf16", residual="rows", pack=True, name="q8_1x10240x10240_bf16"),
        # a short batch of text tokens into the 1280-channel layer, 32-bit results, odd inner width
        _q8("q8_fwd", 77, 1285, 1280, "gelu_tanh", "f32", "f32", name="q8_77x1285x1280_f32"),
        # a wide feed forward's first product in training, z kept in 8 bits: the largest, bound by the matrix cores
        _q8("q8_fwd", 16384, 2560, 10240, "gelu", "bf16", "bf16", z="q8", name="q8_16384x2560x10240_bf16"),
        # training the feed forward of the 640-channel layer from what was kept in 8 bits
        _q8("q8_bwd", 8192, 640, 2560, "gelu", "bf16", "bf16", z="q8", name="q8_bwd_8192x640x2560_bf16"),
        # the same at odd sizes in 32 bits, z kept as it was
        _q8("q8_bwd", 1001, 333, 515, "silu", "f32", "f32", z="full", name="q8_bwd_1001x333x515_f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """Spread over the logarithm; half of the larger ones multiples of 8 or 64, as layers mostly are."""
    v = _log_int(rng, lo, hi)
    r = rng.random()
    if v >= 64 and r < 0.25:
        v -= v % 64
    elif v >= 8 and r < 0.5:
        v -= v % 8
    return v


def draw(rng):
    while True:
        op = rng.choice(["rms_fwd", "rms_bwd", "pack", "q8_fwd", "q8_fwd", "q8_bwd"])
        x_dtype, y_dtype = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
        rows = _size(rng, 1, 16384)
        if op in ("rms_fwd", "rms_bwd", "pack"):
            C = _size(rng, 16, 10240)
            x_stride = C + rng.choice([1, 8, 64]) if rng.random() < 0.15 else 0
            if op == "pack":
                case = _pack(rows, C, rng.choice([0, 0, 32, 64, 128]), x_dtype, x_stride=x_stride)
            else:
                q8 = op == "rms_fwd" and rng.random() < 0.6
                case = _rms(op, rows, C, x_dtype, "bf16" if q8 else y_dtype, residual=op == "rms_fwd" and rng.random() < 0.6, q8=q8,
                            dh=op == "rms_bwd" and rng.random() < 0.6, x_stride=x_stride)
            ok = rows * C <= MAX_VALUES
        else:
            Cin, Cout = _size(rng, 4, 10240), _size(rng, 4, 10240)
            act = rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"])
            y_stride = Cout + rng.choice([1, 8, 64]) if rng.random() < 0.15 else 0
            residual, pixels, z, pack = "none", 0, "none", False
            if op == "q8_fwd":
                residual, pack = rng.choice(["none", "rows", "planar"]), rng.random() < 0.4
                if residual == "planar":
                    pixels = _log_int(rng, 1, rows)
                    rows = pixels * max(1, rows // pixels)
                if act != "none":
                    z = rng.choice(["none", "q8", "full"])
            elif act != "none":
                z = rng.choice(["q8", "full"])
            case = _q8(op, rows, Cin, Cout, act, x_dtype, y_dtype, bias=rng.random() < 0.7, residual=residual, pixels=pixels, z=z,
                       pack=pack, y_stride=y_stride)
            ok = rows * Cin * Cout * (1 if op == "q8_fwd" else 2) <= MAX_PRODUCT
        if ok:
            return case


# ------------------------------------------------------------------- inputs
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, C):
    """Heavy-tailed values (Student's t, 5 degrees of freedom, unit variance), one channel in 64 eight times as large:
    what 8 bits a token have to hold in a transformer's stream."""
    chi = torch.zeros(rows, C, device="cuda")
    for _ in range(5):
        chi += _normal(g, rows, C).square_()
    loud = 1.0 + 7.0 * (torch.rand(C, generator=g, device="cuda") < 1 / 64)
    return _normal(g, rows, C).mul_(math.sqrt(3.0)).div_(chi.sqrt_()).mul_(loud)


def _strided(t, stride, dtype):
    """`t` in rows of `stride` elements, as a slice of a wider tensor."""
    if not stride:
        return t.to(dtype).contiguous()
    wide = torch.zeros(t.shape[:-1] + (stride,), device=t.device, dtype=dtype)
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


def _pad(codes):
    """Codes in rows of whole 128 bytes, zeros behind the last one."""
    return torch.nn.functional.pad(codes, (0, -codes.shape[1] % 128)).to(torch.int8).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"].startswith("rms"):
        return _prepare_rms(case, g)
    return _prepare_pack(case, g) if case["op"] == "pack" else _prepare_q8(case, g)


def _prepare_rms(case, g):
    rows, C = case["rows"], case["C"]
    xt, yt = DTYPES[case["x_dtype"]], DTYPES[case["y_dtype"]]
    s = dict(case=case, gamma=1.0 + 0.1 * _normal(g, C), residual=None, dh=None)
    x = _strided(_activations(g, rows, C), case["x_stride"], xt)
    if case["op"] == "rms_fwd":
        s["x"] = x
        if case["residual"]:
            s["residual"] = _strided(2.0 * _activations(g, rows, C), case["x_stride"], xt)
    else:  # the stream and what the forward pass kept
        s["h"], s["rstd"] = x, (x.double().square().mean(1) + EPS).rsqrt().float()
        s["dy"] = _normal(g, rows, C).to(yt)
        if case["dh"]:
            s["dh"] = _strided(_normal(g, rows, C), case["x_stride"], xt)
    if own:
        import quantized_convolution_amd as q

        p = q.RmsPlan(rows, C, eps=EPS, x_dtype=xt, y_dtype=yt, x_stride=case["x_stride"])
        s["plan"] = p
        if case["op"] == "rms_fwd":
            s["y"], s["rstd"], s["workspace"] = p.empty_output(), p.empty_rstd(), p.empty_workspace()
            s["hbuf"] = p.empty_input() if case["residual"] else None
            if case["q8"]:
                s["codes"], s["scales"] = p.empty_codes()
                s["unpack"] = q.QuantPlan(rows, C, x_dtype=yt)
        else:
            s["dx"], s["dgamma"], s["workspace"] = p.empty_input(), torch.empty_like(s["gamma"]), p.empty_backward_workspace()
    return s


def _prepare_pack(case, g):
    rows, C, xt = case["rows"], case["C"], DTYPES[case["x_dtype"]]
    s = dict(case=case, x=_strided(_activations(g, rows, C), case["x_stride"], xt))
    if own:
        import quantized_convolution_amd as q

        s["plan"] = p = q.QuantPlan(rows, C, group=case["group"], x_dtype=xt, x_stride=case["x_stride"])
        s["codes"], s["scales"] = p.empty_codes()
        s["out"] = p.empty_input()
    return s


def _prepare_q8(case, g):
    M, K, N = case["rows"], case["Cin"], case["Cout"]
    xt, yt = DTYPES[case["x_dtype"]], DTYPES[case["y_dtype"]]
    wq, sw = _to_codes(_normal(g, N, K) / math.sqrt(K))
    s = dict(case=case, wq=_pad(wq), sw=sw, bias=0.1 * _normal(g, N) if case["bias"] else None, residual=None)
    x = _activations(g, M, K)
    if case["pack"]:
        s["x"] = x.to(xt)
    else:
        xq, s["sx"] = _to_codes(x.to(xt).float())
        s["xq"] = _pad(xq)
    del x
    if case["residual"] == "rows":
        s["residual"] = _normal(g, M, N).to(yt)
    elif case["residual"] == "planar":
        s["residual"] = _normal(g, M // case["pixels"], N, case["pixels"]).to(yt)
    if case["op"] == "q8_bwd":
        if case["act"] != "none":  # what the forward pass kept
            z = (s["xq"][:, :K].float() @ wq.float().T) * s["sx"][:, None] * sw
            z = z if s["bias"] is None else z + s["bias"]
            if case["z"] == "q8":
                zq, s["sz"] = _to_codes(z, Z_GROUP)
                s["zq"] = _pad(zq)
            else:
                s["z"] = z.to(yt)
        # one token in eight is padding, whose loss does not count
        dy = _normal(g, M, N) * (torch.rand(M, 1, generator=g, device="cuda") >= 1 / 8)
        s["dy"] = _strided(dy, case["y_stride"], yt)
    if own:
        import quantized_convolution_amd as q

        p = q.Q8LinearPlan(M, K, N, act=case["act"], x_dtype=xt, y_dtype=yt, y_stride=case["y_stride"],
                           r_layout="nchw" if case["residual"] == "planar" else "nhwc", pixels=case["pixels"])
        s["plan"] = p
        if case["op"] == "q8_fwd":
            s["y"], s["workspace"] = p.empty_output(), p.empty_workspace()
            if case["pack"]:
                s["packer"] = q.QuantPlan(M, K, x_dtype=xt)
                s["xq"], s["sx"] = s["packer"].empty_codes()
            if case["z"] == "q8":
                s["zq"], s["sz"] = p.empty_z_codes()
                s["unpack"] = q.QuantPlan(M, N, group=Z_GROUP, x_dtype=torch.bfloat16)
                s["zout"] = s["unpack"].empty_input()
            elif case["z"] == "full":
                s["zbuf"] = p.empty_z()
        else:
            s["dx"], s["dw"], s["workspace"] = p.empty_input(), p.empty_weight_gradient(), p.empty_backward_workspace()
            s["dbias"] = torch.empty_like(s["bias"]) if case["bias"] else None
    return s


# --------------------------------------------------------------- plain forms
def _to_codes(x, group=0):
    """Codes (whole numbers in 32-bit floats) and scales of rows, or of groups of columns: the largest magnitude of
    each becomes 127. Quotients are of tensors: with a number torch multiplies by a rounded reciprocal."""
    rows, C = x.shape
    n = group or C
    v = torch.nn.functional.pad(x, (0, -C % n)).reshape(rows, -1, n)
    a = v.abs().amax(dim=2, keepdim=True)
    most = torch.full_like(a, 127.0)
    codes = torch.round(v * torch.where(a > 0, most / a, torch.zeros_like(a)))
    codes, scales = codes.reshape(rows, -1)[:, :C], (a / most)[:, :, 0]
    return codes, (scales if group else scales[:, 0])


def _values(codes, scales, group=0):
    """What codes stand for, in 32 bits."""
    if not group:
        return codes * scales[:, None]
    return codes * scales.repeat_interleave(group, dim=1)[:, :codes.shape[1]]


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_rms_fwd(s):
    c = s["case"]
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(DTYPES[c["x_dtype"]])
    v = h.float()
    rstd = 1 / torch.sqrt((v * v).mean(dim=1) + EPS)
    if c["q8"]:  # the norm's factor is the same for a whole row: it is in the scale alone
        codes, scales = _to_codes(v * s["gamma"])
        y = _values(codes, scales * rstd)
    else:
        y = v * rstd[:, None] * s["gamma"]
    out = {"y": y.to(DTYPES[c["y_dtype"]]), "rstd": rstd}
    if s["residual"] is not None:
        out["h"] = h
    return out


def _plain_rms_bwd(s):
    c = s["case"]
    n = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    t = dy * s["gamma"]
    dx = s["rstd"][:, None] * (t - n * (t * n).mean(dim=1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(DTYPES[c["x_dtype"]]), "dgamma": (dy * n).sum(dim=0)}


def _plain_pack(s):
    codes, scales = _to_codes(s["x"].float(), s["case"]["group"])
    return {"x": _values(codes, scales, s["case"]["group"]).to(DTYPES[s["case"]["x_dtype"]]), "scales": scales}


def _plain_q8_fwd(s):
    c = s["case"]
    yt = DTYPES[c["y_dtype"]]
    if c["pack"]:
        xq, sx = _to_codes(s["x"].float())
    else:
        xq, sx = s["xq"][:, :c["Cin"]].float(), s["sx"]
    z = (xq @ s["wq"][:, :c["Cin"]].float().T) * sx[:, None] * s["sw"]
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, c["act"])
    if c["residual"] == "rows":
        y = y + s["residual"].float()
    elif c["residual"] == "planar":
        y = y + s["residual"].float().permute(0, 2, 1).reshape(y.shape)
    out = {"y": y.to(yt)}
    if c["z"] == "full":
        out["z"] = z.to(yt)
    elif c["z"] == "q8":
        out["z"] = _values(*_to_codes(z, Z_GROUP), Z_GROUP).to(torch.bfloat16)
    return out


def _plain_q8_bwd(s):
    c = s["case"]
    dz = s["dy"].float()
    if c["act"] != "none":
        z = _values(s["zq"][:, :c["Cout"]].float(), s["sz"], Z_GROUP) if c["z"] == "q8" else s["z"].float()
        dz = dz * _act_slope(z, c["act"])
    xt = DTYPES[c["x_dtype"]]
    w = s["wq"][:, :c["Cin"]].float() * s["sw"][:, None]
    x = s["xq"][:, :c["Cin"]].float() * s["sx"][:, None]
    out = {"dx": (dz @ w).to(xt), "dw": (dz.T @ x).to(xt)}
    if c["bias"]:
        out["dbias"] = dz.sum(dim=0)
    return out


# --------------------------------------------------------- the framework's
def _own_rms_fwd(s):
    import quantized_convolution_amd as q

    if s["case"]["q8"]:
        q.wq8_rms_forward(s["plan"], s["x"], s["gamma"], s["residual"], h=s["hbuf"], codes=s["codes"], scales=s["scales"],
                          rstd=s["rstd"], want_y=False, workspace=s["workspace"])
        q.wq8_quant_unpack(s["unpack"], s["codes"], s["scales"], x=s["y"])
    else:
        q.wq8_rms_forward(s["plan"], s["x"], s["gamma"], s["residual"], y=s["y"], h=s["hbuf"], rstd=s["rstd"],
                          workspace=s["workspace"])
    out = {"y": s["y"], "rstd": s["rstd"]}
    return dict(out, h=s["hbuf"]) if s["hbuf"] is not None else out


def _own_rms_bwd(s):
    import quantized_convolution_amd as q

    q.wq8_rms_backward(s["plan"], s["dy"], s["h"], s["rstd"], s["gamma"], dh=s["dh"], dx=s["dx"], dgamma=s["dgamma"],
                       workspace=s["workspace"])
    return {"dx": s["dx"], "dgamma": s["dgamma"]}


def _own_pack(s):
    import quantized_convolution_amd as q

    q.wq8_quant_pack(s["plan"], s["x"], codes=s["codes"], scales=s["scales"])
    q.wq8_quant_unpack(s["plan"], s["codes"], s["scales"], x=s["out"])
    return {"x": s["out"], "scales": s["scales"]}


def _own_q8_fwd(s):
    import quantized_convolution_amd as q

    if s["case"]["pack"]:
        q.wq8_quant_pack(s["packer"], s["x"], codes=s["xq"], scales=s["sx"])
    args = (s["plan"], s["xq"], s["sx"], s["wq"], s["sw"], s["bias"], s["residual"])
    if s["case"]["z"] == "q8":
        q.wq8_q8linear_forward(*args, y=s["y"], zq=s["zq"], sz=s["sz"], workspace=s["workspace"])
        return {"y": s["y"], "z": q.wq8_quant_unpack(s["unpack"], s["zq"], s["sz"], x=s["zout"])}
    if s["case"]["z"] == "full":
        q.wq8_q8linear_forward(*args, y=s["y"], z=s["zbuf"], workspace=s["workspace"])
        return {"y": s["y"], "z": s["zbuf"]}
    return {"y": q.wq8_q8linear_forward(*args, y=s["y"], workspace=s["workspace"])}


def _own_q8_bwd(s):
    import quantized_convolution_amd as q

    q.wq8_q8linear_backward(s["plan"], s["dy"], s["xq"], s["sx"], s["wq"], s["sw"], z=s.get("z"), zq=s.get("zq"), sz=s.get("sz"),
                            dx=s["dx"], dw=s["dw"], dbias=s["dbias"], workspace=s["workspace"])
    return {k: s[k] for k in ("dx", "dw", "dbias") if s[k] is not None}


PLAIN = {"rms_fwd": _plain_rms_fwd, "rms_bwd": _plain_rms_bwd, "pack": _plain_pack, "q8_fwd": _plain_q8_fwd,
         "q8_bwd": _plain_q8_bwd}
OWN = {"rms_fwd": _own_rms_fwd, "rms_bwd": _own_rms_bwd, "pack": _own_pack, "q8_fwd": _own_q8_fwd, "q8_bwd": _own_q8_bwd}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits
ACT64 = {"none": lambda z: z * 1.0, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}


def _codes64(v, group):
    """The whole numbers that values are held by, and the scales. Which of two neighbours a value of 32 bits goes to is
    part of the definition: it is multiplied by 127 / a, both rounded to 32 bits."""
    at = (torch.arange(v.shape[1], device=v.device) // (group or v.shape[1])).expand(v.shape)
    a = v.new_zeros(v.shape[0], int(at[0, -1]) + 1).scatter_reduce_(1, at, v.abs(), "amax")
    f = torch.full_like(a, 127.0).div_(a).masked_fill_(a == 0, 0.0)
    return v.mul(f.gather(1, at)).round_().double(), a.double() / 127


def _stands_for(codes, scales, group):
    at = torch.arange(codes.shape[1], device=codes.device) // (group or codes.shape[1])
    return codes * scales[:, at]


def exact(case, seed):
    s = prepare(case, seed)
    f64 = lambda t: t.detach().double()  # noqa: E731
    if case["op"] == "rms_fwd":
        x = f64(s["x"])
        if s["residual"] is not None:  # the stream is held in x's type
            x = (x + f64(s["residual"])).float().to(DTYPES[case["x_dtype"]]).double()
        rstd = (x.square().mean(1) + EPS) ** -0.5
        y = x * s["gamma"].double()
        if case["q8"]:
            codes, scales = _codes64(y, 0)
            y = _stands_for(codes, scales, 0)
        out = {"y": y * rstd[:, None], "rstd": rstd}
        return dict(out, h=x) if s["residual"] is not None else out
    if case["op"] == "rms_bwd":
        h, gamma = f64(s["h"]).requires_grad_(), f64(s["gamma"]).requires_grad_()
        with torch.enable_grad():
            y = h * (h.square().mean(1, keepdim=True) + EPS) ** -0.5 * gamma
            dx, dgamma = torch.autograd.grad(y, (h, gamma), f64(s["dy"]))
        return {"dx": dx if s["dh"] is None else dx + f64(s["dh"]), "dgamma": dgamma}
    if case["op"] == "pack":
        codes, scales = _codes64(s["x"].float(), case["group"])
        return {"x": _stands_for(codes, scales, case["group"]), "scales": scales if case["group"] else scales[:, 0]}
    K, N = case["Cin"], case["Cout"]
    w = s["wq"][:, :K].double() * f64(s["sw"])[:, None]
    if case["pack"]:
        x = _stands_for(*_codes64(s["x"].float(), 0), 0)
    else:
        x = s["xq"][:, :K].double() * f64(s["sx"])[:, None]
    if case["op"] == "q8_fwd":
        b = torch.zeros(N, device=x.device, dtype=torch.float64) if s["bias"] is None else f64(s["bias"])
        z = torch.addmm(b, x, w.t())
        y = ACT64[case["act"]](z)
        if case["residual"] == "rows":
            y = y + f64(s["residual"])
        elif case["residual"] == "planar":
            y = (y.reshape(-1, case["pixels"], N) + f64(s["residual"]).transpose(1, 2)).reshape(z.shape)
        if case["z"] == "none":
            return {"y": y}
        return {"y": y, "z": z if case["z"] == "full" else _stands_for(*_codes64(z, Z_GROUP), Z_GROUP)}
    dz = f64(s["dy"])
    if case["act"] != "none":
        z = _stands_for(s["zq"][:, :N].double(), f64(s["sz"]), Z_GROUP) if case["z"] == "q8" else f64(s["z"])
        z.requires_grad_()
        with torch.enable_grad():
            dz = torch.autograd.grad(ACT64[case["act"]](z), z, dz)[0]
    out = {"dx": dz.mm(w), "dw": dz.t().mm(x)}
    if case["bias"]:
        out["dbias"] = dz.sum(0)
    return out


# ------------------------------------------------------------------- work
def work(case):
    size = {"f32": 4, "bf16": 2}
    xs = size[case["x_dtype"]]
    if case["op"] == "pack":  # x in, the values that its codes stand for and the scales out
        n, scales = case["rows"] * case["C"], case["rows"] * -(-case["C"] // (case["group"] or case["C"]))
        return {"bytes": 2 * n * xs + 4 * scales, "flops": 4 * n}
    ys = size[case["y_dtype"]]
    if case["op"].startswith("rms"):
        n, small = case["rows"] * case["C"], 4 * (case["rows"] + case["C"])
        if case["op"] == "rms_fwd":  # x (and the residual in, the stream out), y out
            return {"bytes": n * (xs * (3 if case["residual"] else 1) + ys) + small, "flops": 8 * n}
        return {"bytes": n * (xs * (3 if case["dh"] else 2) + ys) + small + 4 * case["C"], "flops": 10 * n}
    M, K, N = case["rows"], case["Cin"], case["Cout"]
    small = 4 * N * (1 + case["bias"]) + 4 * M
    if case["op"] == "q8_fwd":
        outs = 1 + (case["residual"] != "none") + (case["z"] == "full")
        x = M * K * (xs if case["pack"] else 1)
        return {"bytes": x + N * K + ys * M * N * outs + 2 * M * N * (case["z"] == "q8") + small, "flops": 2 * M * K * N}
    z = 0 if case["act"] == "none" else M * N * ys if case["z"] == "full" else M * N + 4 * M * -(-N // Z_GROUP)
    return {"bytes": (1 + xs) * (M * K + N * K) + ys * M * N + z + small, "flops": 4 * M * K * N}
