"""Cases for the group norm and the matrix product that stand around the
framework's convolutions in a UNet, forward and backward.

`listed()` gives named cases, `draw(rng)` further ones of the same ranges.
`prepare` makes a case's inputs from a seed, `run` makes one pass: with `own`
set through the framework's entry points, else in plain torch operations in
32 bits. `exact` evaluates the definitions in 64 bits, `work` counts the bytes
and operations that a pass cannot do without.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5

# Cost bounds of drawn cases: the largest listed ones (elements normalised,
# multiply-adds of one product).
MAX_NORM = 8 * 640 * 128 * 128
MAX_PRODUCT = 16384 * 2560 * 10240


def _norm(op, N, C, H, W, act, x_dtype, y_dtype, x_layout, y_layout, groups=32, shift=False, x_stride=0, name=None):
    case = dict(op=op, N=N, C=C, H=H, W=W, groups=groups, act=act, x_dtype=x_dtype, y_dtype=y_dtype,
                x_layout=x_layout, y_layout=y_layout, shift=shift, x_stride=x_stride)
    return dict(case, name=name) if name else case


def _linear(op, rows, Cin, Cout, act, x_dtype, y_dtype, bias=True, residual="none", pixels=0, z=False, x_stride=0,
            y_stride=0, name=None):
    case = dict(op=op, rows=rows, Cin=Cin, Cout=Cout, act=act, x_dtype=x_dtype, y_dtype=y_dtype, bias=bias,
                residual=residual, pixels=pixels, z=z, x_stride=x_stride, y_stride=y_stride)
    return dict(case, name=name) if name else case


def listed():
    return [
        # the norm after the time embedding's addition, between the two convolutions of a block: NCHW in and out
        _norm("norm_fwd", 8, 1280, 16, 16, "silu", "f32", "f32", "nchw", "nchw", shift=True, name="norm_c1280_16x16_f32_nchw"),
        # the last ResNet-18 stage's size in bfloat16: many small images, short groups
        _norm("norm_fwd", 32, 512, 7, 7, "relu", "bf16", "bf16", "nhwc", "nhwc", name="norm_c512_7x7_bf16"),
        # a block's first norm: channels-last stream in, NCHW out for the convolution
        _norm("norm_fwd", 2, 320, 64, 64, "silu", "bf16", "bf16", "nhwc", "nchw", name="norm_c320_64x64_bf16_to_nchw"),
        # a decoder at twice the UNet's resolution, the largest: bound by memory
        _norm("norm_fwd", 8, 640, 128, 128, "silu", "bf16", "bf16", "nhwc", "nhwc", name="norm_c640_128x128_bf16"),
        # training at the 640-channel layer
        _norm("norm_bwd", 8, 640, 32, 32, "silu", "bf16", "bf16", "nhwc", "nhwc", name="norm_bwd_c640_32x32_bf16"),
        # training in 32 bits, gradient arriving in NCHW from the convolution's side, time embedding's gradient too
        _norm("norm_bwd", 2, 320, 64, 64, "silu", "f32", "f32", "nhwc", "nchw", shift=True, name="norm_bwd_c320_64x64_f32_nchw"),
        # the time embedding's projection, one row for each of 8 images: latency of a single-token product
        _linear("linear_fwd", 8, 320, 1280, "silu", "bf16", "bf16", name="linear_8x320x1280_bf16"),
        # the token projection of the 640-channel layer with its residual
        _linear("linear_fwd", 8192, 640, 640, "none", "bf16", "bf16", residual="rows", name="linear_8192x640x640_bf16"),
        # a decoder block's 1x1 shortcut over a concatenated stream, the convolution's NCHW output as residual, 32 bits
        _linear("linear_fwd", 2048, 2560, 1280, "none", "f32", "f32", residual="planar", pixels=256, name="linear_2048x2560x1280_f32"),
        # a wide feed forward's first product over many tokens, the largest: bound by the matrix cores
        _linear("linear_fwd", 16384, 2560, 10240, "gelu", "bf16", "bf16", name="linear_16384x2560x10240_bf16"),
        # training the feed forward of the 640-channel layer
        _linear("linear_bwd", 8192, 640, 2560, "gelu", "bf16", "bf16", name="linear_bwd_8192x640x2560_bf16"),
        # training at odd sizes in 32 bits: no row starts on a vector's boundary
        _linear("linear_bwd", 1001, 333, 515, "silu", "f32", "f32", name="linear_bwd_1001x333x515_f32"),
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
        op = rng.choice(["norm_fwd", "norm_bwd", "linear_fwd", "linear_bwd"])
        dtypes = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
        if op.startswith("norm"):
            # relu's gradient jumps where the last bit of z decides its sign, so it is not drawn for the backward pass
            act = rng.choice(["none", "silu", "gelu", "gelu_tanh"] + (["relu"] if op == "norm_fwd" else []))
            groups = rng.choice([1, 2, 4, 8, 16, 32, 32])
            C = groups * _log_int(rng, 1, 80)
            N, H, W = _log_int(rng, 1, 32), _log_int(rng, 1, 128), _log_int(rng, 1, 128)
            x_layout, y_layout = rng.choice(["nhwc", "nhwc", "nchw"]), rng.choice(["nhwc", "nhwc", "nchw"])
            x_stride = C + rng.choice([1, 8, 64]) if x_layout == "nhwc" and rng.random() < 0.15 else 0
            case = _norm(op, N, C, H, W, act, *dtypes, x_layout, y_layout, groups=groups, shift=rng.random() < 0.3, x_stride=x_stride)
            # a group of a few values has a gradient that is nothing but what its terms leave
            ok = N * C * H * W <= MAX_NORM and C // groups * H * W >= 16
        else:
            act = rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"])
            Cin, Cout = _size(rng, 4, 10240), _size(rng, 4, 10240)
            residual, pixels = (rng.choice(["none", "rows", "planar"]), 0) if op == "linear_fwd" else ("none", 0)
            rows = _size(rng, 1, 16384)
            if residual == "planar":
                pixels = _log_int(rng, 1, rows)
                rows = pixels * max(1, rows // pixels)
            x_stride = Cin + rng.choice([1, 8, 64]) if rng.random() < 0.15 else 0
            y_stride = Cout + rng.choice([1, 8, 64]) if rng.random() < 0.15 else 0
            case = _linear(op, rows, Cin, Cout, act, *dtypes, bias=rng.random() < 0.7, residual=residual, pixels=pixels,
                           z=op == "linear_fwd" and act != "none" and rng.random() < 0.3, x_stride=x_stride, y_stride=y_stride)
            ok = rows * Cin * Cout * (1 if op == "linear_fwd" else 2) <= MAX_PRODUCT
        if ok and 3072 not in case.values():
            return case


# ------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, *shape):
    """Heavy-tailed values (Student's t, 5 degrees of freedom, unit variance), as UNet activations are."""
    chi = torch.zeros(shape, device="cuda")
    for _ in range(5):
        chi += _normal(g, *shape).square_()
    return _normal(g, *shape).mul_(math.sqrt(3.0)).div_(chi.sqrt_())


def _strided(t, stride, dtype):
    """`t` (last dimension contiguous) in rows of `stride` elements, as a slice of a wider tensor."""
    if not stride:
        return t.to(dtype).contiguous()
    wide = torch.zeros(t.shape[:-1] + (stride,), device=t.device, dtype=dtype)
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


def _to_layout(t, layout):
    """[N, H, W, C] -> a contiguous tensor of the layout."""
    return (t if layout == "nhwc" else t.permute(0, 3, 1, 2)).contiguous()


def _from_layout(t, layout):
    """The [N, H, W, C] view of a tensor of the layout."""
    return t if layout == "nhwc" else t.permute(0, 2, 3, 1)


def prepare(case, seed):
    g = _generator(seed)
    return (_prepare_norm if case["op"].startswith("norm") else _prepare_linear)(case, g)


def _prepare_norm(case, g):
    N, C, H, W, G = (case[k] for k in ("N", "C", "H", "W", "groups"))
    xt, yt = DTYPES[case["x_dtype"]], DTYPES[case["y_dtype"]]
    x = _activations(g, N, H, W, C) * (1.0 + 0.25 * _normal(g, C)) + 0.5 + 0.5 * _normal(g, C)
    x = _strided(x, case["x_stride"], xt) if case["x_layout"] == "nhwc" else _to_layout(x, "nchw").to(xt)
    s = dict(case=case, x=x, gamma=1.0 + 0.1 * _normal(g, C), beta=0.1 * _normal(g, C),
             shift=0.5 * _normal(g, N, C) if case["shift"] else None)
    v = _from_layout(x, case["x_layout"]).double()
    if case["shift"]:
        v = v + s["shift"].double()[:, None, None, :]
    if case["op"] == "norm_bwd":  # what the forward pass kept
        var, mean = torch.var_mean(v.reshape(N, H * W, G, C // G), dim=(1, 3), correction=0)
        s["mean"], s["rstd"] = mean.float(), (var + EPS).rsqrt().float()
        s["dy"] = _to_layout(_normal(g, N, H, W, C), case["y_layout"]).to(yt)
    if own:
        import quantized_convolution_amd as q

        p = q.NormPlan(N, C, H, W, groups=G, eps=EPS, act=case["act"], x_dtype=xt, y_dtype=yt, x_layout=case["x_layout"],
                       y_layout=case["y_layout"], x_stride=case["x_stride"])
        s["plan"] = p
        if case["op"] == "norm_fwd":
            s["y"], s["workspace"] = p.empty_output(), p.empty_workspace()
            s["mean"], s["rstd"] = p.empty_stats()
        else:
            s["dx"], s["workspace"] = p.empty_input(), p.empty_backward_workspace()
            s["dgamma"], s["dbeta"] = torch.empty_like(s["gamma"]), torch.empty_like(s["beta"])
            s["dshift"] = torch.empty_like(s["shift"]) if case["shift"] else None
    return s


def _prepare_linear(case, g):
    M, K, N = case["rows"], case["Cin"], case["Cout"]
    xt, yt = DTYPES[case["x_dtype"]], DTYPES[case["y_dtype"]]
    x = _strided(_activations(g, M, K), case["x_stride"], xt)
    w = (_normal(g, N, K) / math.sqrt(K)).to(xt)
    s = dict(case=case, x=x, w=w, bias=0.1 * _normal(g, N) if case["bias"] else None, residual=None)
    if case["residual"] == "rows":
        s["residual"] = _activations(g, M, N).to(yt)
    elif case["residual"] == "planar":
        s["residual"] = _activations(g, M // case["pixels"], N, case["pixels"]).to(yt)
    if case["op"] == "linear_bwd":
        s["z"] = None
        if case["act"] != "none":  # what the forward pass kept
            z = x.float() @ w.float().T
            s["z"] = (z if s["bias"] is None else z + s["bias"]).to(yt)
        s["dy"] = _strided(_normal(g, M, N), case["y_stride"], yt)
    if own:
        import quantized_convolution_amd as q

        p = q.LinearPlan(M, K, N, act=case["act"], x_dtype=xt, y_dtype=yt, x_stride=case["x_stride"], y_stride=case["y_stride"],
                         r_layout="nchw" if case["residual"] == "planar" else "nhwc", pixels=case["pixels"])
        s["plan"] = p
        if case["op"] == "linear_fwd":
            s["y"], s["workspace"] = p.empty_output(), p.empty_workspace()
            s["zbuf"] = p.empty_z() if case["z"] else None
        else:
            s["dx"], s["dw"], s["workspace"] = p.empty_input(), torch.empty_like(w), p.empty_backward_workspace()
            s["dbias"] = torch.empty_like(s["bias"]) if case["bias"] else None
    return s


# --------------------------------------------------------------- plain forms
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


def _grouped(t, groups):
    """[N, H, W, C] -> [N, P, groups, C / groups]."""
    N, H, W, C = t.shape
    return t.reshape(N, H * W, groups, C // groups)


def _plain_norm_fwd(s):
    c = s["case"]
    v = _from_layout(s["x"], c["x_layout"]).float()
    if s["shift"] is not None:
        v = v + s["shift"][:, None, None, :]
    shape = v.shape
    v = _grouped(v, c["groups"])
    mean = v.mean(dim=(1, 3), keepdim=True)
    d = v - mean
    rstd = 1 / torch.sqrt((d * d).mean(dim=(1, 3), keepdim=True) + EPS)
    z = (d * rstd).reshape(shape) * s["gamma"] + s["beta"]
    y = _to_layout(_act(z, c["act"]), c["y_layout"]).to(DTYPES[c["y_dtype"]])
    return {"y": y, "mean": mean.reshape(shape[0], -1), "rstd": rstd.reshape(shape[0], -1)}


def _plain_norm_bwd(s):
    c = s["case"]
    v = _from_layout(s["x"], c["x_layout"]).float()
    if s["shift"] is not None:
        v = v + s["shift"][:, None, None, :]
    shape = v.shape
    rstd = s["rstd"][:, None, :, None]
    h = (_grouped(v, c["groups"]) - s["mean"][:, None, :, None]) * rstd
    z = h.reshape(shape) * s["gamma"] + s["beta"]
    dz = _from_layout(s["dy"], c["y_layout"]).float() * _act_slope(z, c["act"])
    t = _grouped(dz * s["gamma"], c["groups"])
    dx = rstd * (t - t.mean(dim=(1, 3), keepdim=True) - h * (t * h).mean(dim=(1, 3), keepdim=True))
    dx = dx.reshape(shape)
    out = {"dx": _to_layout(dx, c["x_layout"]).to(DTYPES[c["x_dtype"]]), "dgamma": (dz * h.reshape(shape)).sum(dim=(0, 1, 2)),
           "dbeta": dz.sum(dim=(0, 1, 2))}
    if s["shift"] is not None:
        out["dshift"] = dx.sum(dim=(1, 2))
    return out


def _plain_linear_fwd(s):
    c = s["case"]
    yt = DTYPES[c["y_dtype"]]
    z = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, c["act"])
    if c["residual"] == "rows":
        y = y + s["residual"].float()
    elif c["residual"] == "planar":
        y = y + s["residual"].float().permute(0, 2, 1).reshape(y.shape)
    out = {"y": y.to(yt)}
    if c["z"]:
        out["z"] = z.to(yt)
    return out


def _plain_linear_bwd(s):
    c = s["case"]
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_slope(s["z"].float(), c["act"])
    xt = DTYPES[c["x_dtype"]]
    out = {"dx": (dz @ s["w"].float()).to(xt), "dw": (dz.T @ s["x"].float()).to(xt)}
    if c["bias"]:
        out["dbias"] = dz.sum(dim=0)
    return out


# --------------------------------------------------------- the framework's
def _own_norm_fwd(s):
    import quantized_convolution_amd as q

    y = q.wq8_norm_forward(s["plan"], s["x"], s["gamma"], s["beta"], shift=s["shift"], y=s["y"], mean=s["mean"], rstd=s["rstd"],
                           workspace=s["workspace"])
    return {"y": y, "mean": s["mean"], "rstd": s["rstd"]}


def _own_norm_bwd(s):
    import quantized_convolution_amd as q

    q.wq8_norm_backward(s["plan"], s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"], s["beta"], shift=s["shift"], dx=s["dx"],
                        dgamma=s["dgamma"], dbeta=s["dbeta"], dshift=s["dshift"], workspace=s["workspace"])
    return {k: s[k] for k in ("dx", "dgamma", "dbeta", "dshift") if s[k] is not None}


def _own_linear_fwd(s):
    import quantized_convolution_amd as q

    y = q.wq8_linear_forward(s["plan"], s["x"], s["w"], s["bias"], s["residual"], y=s["y"], z=s["zbuf"], workspace=s["workspace"])
    return {"y": y, "z": s["zbuf"]} if s["zbuf"] is not None else {"y": y}


def _own_linear_bwd(s):
    import quantized_convolution_amd as q

    q.wq8_linear_backward(s["plan"], s["dy"], s["x"], s["w"], z=s["z"], dx=s["dx"], dw=s["dw"], dbias=s["dbias"],
                          workspace=s["workspace"])
    return {k: s[k] for k in ("dx", "dw", "dbias") if s[k] is not None}


PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "linear_fwd": _plain_linear_fwd, "linear_bwd": _plain_linear_bwd}
OWN = {"norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd, "linear_fwd": _own_linear_fwd, "linear_bwd": _own_linear_bwd}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits
ACT64 = {"none": lambda z: z * 1.0, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}


def _norm64(c, s, leaves):
    """The forward pass in NCHW and 64 bits: y, mean, rstd."""
    N, C, G = c["N"], c["C"], c["groups"]
    v = leaves["x"]
    if "shift" in leaves:
        v = v + leaves["shift"][:, :, None, None]
    var, mean = torch.var_mean(v.reshape(N, G, -1), dim=2, correction=0)
    rstd = (var + EPS) ** -0.5
    h = (v.reshape(N, G, -1) - mean[..., None]) * rstd[..., None]
    return ACT64[c["act"]](h.reshape(v.shape) * leaves["gamma"][:, None, None] + leaves["beta"][:, None, None]), mean, rstd


def exact(case, seed):
    s = prepare(case, seed)
    f64 = lambda t: t.detach().double()  # noqa: E731
    if case["op"].startswith("norm"):
        nchw = lambda t, layout: f64(t if layout == "nchw" else t.permute(0, 3, 1, 2))  # noqa: E731
        back = lambda t, layout: t if layout == "nchw" else t.permute(0, 2, 3, 1)  # noqa: E731
        leaves = {"x": nchw(s["x"], case["x_layout"]), "gamma": f64(s["gamma"]), "beta": f64(s["beta"])}
        if s["shift"] is not None:
            leaves["shift"] = f64(s["shift"])
        if case["op"] == "norm_fwd":
            y, mean, rstd = _norm64(case, s, leaves)
            return {"y": back(y, case["y_layout"]), "mean": mean, "rstd": rstd}
        leaves = {k: v.requires_grad_() for k, v in leaves.items()}
        with torch.enable_grad():
            y = _norm64(case, s, leaves)[0]
            grads = dict(zip(leaves, torch.autograd.grad(y, list(leaves.values()), nchw(s["dy"], case["y_layout"]))))
        grads["x"] = back(grads["x"], case["x_layout"])
        return {"d" + k: v for k, v in grads.items()}
    x, w = f64(s["x"]), f64(s["w"])
    if case["op"] == "linear_fwd":
        b = torch.zeros(case["Cout"], device=x.device, dtype=torch.float64) if s["bias"] is None else f64(s["bias"])
        z = torch.addmm(b, x, w.t())
        y = ACT64[case["act"]](z)
        if case["residual"] == "rows":
            y = y + f64(s["residual"])
        elif case["residual"] == "planar":
            y = (y.reshape(-1, case["pixels"], case["Cout"]) + f64(s["residual"]).transpose(1, 2)).reshape(z.shape)
        return {"y": y, "z": z} if case["z"] else {"y": y}
    dz = f64(s["dy"])
    if s["z"] is not None:
        z = f64(s["z"]).requires_grad_()
        with torch.enable_grad():
            dz = torch.autograd.grad(ACT64[case["act"]](z), z, dz)[0]
    out = {"dx": dz.mm(w), "dw": dz.t().mm(x)}
    if case["bias"]:
        out["dbias"] = dz.sum(0)
    return out


# ------------------------------------------------------------------- work
def work(case):
    size = {"f32": 4, "bf16": 2}
    xs, ys = size[case["x_dtype"]], size[case["y_dtype"]]
    if case["op"].startswith("norm"):
        n = case["N"] * case["C"] * case["H"] * case["W"]
        params = 4 * (2 * case["C"] + 2 * case["N"] * case["groups"] + (case["N"] * case["C"] if case["shift"] else 0))
        if case["op"] == "norm_fwd":  # x in, y out, statistics out
            return {"bytes": n * (xs + ys) + params, "flops": 10 * n}
        return {"bytes": n * (2 * xs + ys) + 2 * params, "flops": 25 * n}  # x and dy in, dx out
    M, K, N = case["rows"], case["Cin"], case["Cout"]
    if case["op"] == "linear_fwd":
        outs = 1 + (case["residual"] != "none") + case["z"]
        return {"bytes": xs * (M * K + N * K) + ys * M * N * outs + 4 * N * case["bias"], "flops": 2 * M * K * N}
    ins = 1 + (case["act"] != "none")  # dy, z
    return {"bytes": 2 * xs * (M * K + N * K) + ys * M * N * ins + 4 * N * case["bias"], "flops": 4 * M * K * N}
