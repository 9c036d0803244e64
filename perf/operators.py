"""The Linear epilogue and layer-norm operators of the FP8 stack as measured workloads.

Four operators: the FP8 Linear with bias, activation and residual in its
epilogue, that epilogue's backward pass, the layer norm and its backward
pass.  ``run`` computes a case in plain torch operations in 32 bits, or, with
``own`` true, through ``mlp_fp8_quant_amd``; ``exact`` is the definition in 64
bits.  FP8 results are returned as float8 values.
"""

import math

import torch

own = False

EPS = 1e-5
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _linear(name, m, n, k, act, bias, residual, out, rowwise=False, pre=False):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "act": act, "bias": bias,
            "residual": residual, "out": out, "rowwise": rowwise, "pre": pre}


def _linear_bwd(name, m, n, act):
    return {"name": name, "op": "linear_bwd", "m": m, "n": n, "act": act}


def _norm(name, m, h, x, w, out, stats):
    return {"name": name, "op": "norm", "m": m, "h": h, "x": x, "w": w, "out": out, "stats": stats}


def _norm_bwd(name, m, h, x, dy, w, dres):
    return {"name": name, "op": "norm_bwd", "m": m, "h": h, "x": x, "dy": dy, "w": w, "dres": dres}


def listed():
    return [
        # one token through the decoder layer's o projection, added to the residual stream
        _linear("linear token o", 1, 4096, 4096, "none", "bf16", "bf16", "bf16"),
        # a small odd batch of tokens through an up projection whose output the next Linear reads as FP8
        _linear("linear 13 tokens up", 13, 12288, 4096, "gelu", "f32", "none", "fp8"),
        # the understanding tower's down projection (512 tokens) with its residual
        _linear("linear 512 tokens down", 512, 4096, 12288, "none", "none", "bf16", "bf16"),
        # training forward at sizes no tile divides: per-token / per-channel scales, a 32-bit residual
        # stream, the pre-activation kept for the backward pass
        _linear("linear ragged training", 777, 2053, 2064, "silu", "f32", "f32", "f32", True, True),
        # the large tower's up projection, FP8 out
        _linear("linear large up", 16384, 25600, 5120, "gelu_tanh", "bf16", "none", "fp8"),
        # backward of the epilogue: a ragged batch, and the generation tower's up projection
        _linear_bwd("linear backward ragged", 777, 2053, "silu"),
        _linear_bwd("linear backward gen up", 4096, 12288, "gelu_tanh"),
        # the norm of one token before its quantized projections
        _norm("norm token", 1, 4096, "bf16", "bf16", "fp8", False),
        # training forward of an odd width from a 32-bit residual stream
        _norm("norm ragged training", 1531, 1027, "f32", "f32", "bf16", True),
        # the large tower's norm, FP8 codes straight to its Linears
        _norm("norm large", 16384, 5120, "bf16", "bf16", "fp8", False),
        # backward at the understanding tower's size, and at the large tower's with the residual's gradient added
        _norm_bwd("norm backward 512 tokens", 512, 4096, "bf16", "bf16", "f32", False),
        _norm_bwd("norm backward large", 16384, 5120, "bf16", "bf16", "bf16", True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "norm", "norm_bwd"])
    if op == "linear":
        c = _linear("", _log(rng, 1, 6000), _log(rng, 64, 16384), 16 * _log(rng, 16, 768),
                    rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                    rng.choice(["none", "bf16", "f32"]), rng.choice(["none", "bf16", "f32"]),
                    rng.choice(["bf16", "bf16", "fp8", "f32"]))
        c["rowwise"] = c["out"] != "fp8" and rng.random() < 0.3
        c["pre"] = rng.random() < 0.2
    elif op == "linear_bwd":
        c = _linear_bwd("", _log(rng, 1, 6000), _log(rng, 64, 16384),
                        rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]))
    elif op == "norm":
        c = _norm("", _log(rng, 1, 12000), _log(rng, 32, 8192), rng.choice(["bf16", "f32"]),
                  rng.choice(["bf16", "f32"]), rng.choice(["bf16", "fp8", "f32"]), rng.random() < 0.5)
    else:
        c = _norm_bwd("", _log(rng, 1, 12000), _log(rng, 32, 8192), rng.choice(["bf16", "f32"]),
                      rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]), rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _acts(gen, rows, cols):
    """N(0, 1) with 0.5% of the entries times 20."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    return torch.where(torch.rand(rows, cols, generator=gen, device="cuda") < 0.005, 20.0 * x, x)


def _codes(x, rowwise):
    """E4M3 codes of x and their scale(s), amax / 448 over the tensor or over each row."""
    amax = x.abs().amax(dim=1) if rowwise else x.abs().amax().reshape(1)
    s = amax / 448.0
    q = (x / (s[:, None] if rowwise else s)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    s = {"case": case}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s["qx"], s["sx"] = _codes(_acts(gen, m, k).to(torch.bfloat16).float(), case["rowwise"])
        s["qw"], s["sw"] = _codes((0.02 * randn(n, k)).to(torch.bfloat16).float(), case["rowwise"])
        s["bias"] = None if case["bias"] == "none" else (0.1 * randn(n)).to(_TYPES[case["bias"]])
        s["residual"] = None if case["residual"] == "none" else _acts(gen, m, n).to(_TYPES[case["residual"]])
        # a calibrated output scale: about the largest value that a projection of such inputs gives
        s["sy"] = torch.full((1,), 0.02 * math.sqrt(k) * 8.0 / 448.0 + 0.01, device="cuda") \
            if case["out"] == "fp8" else None
    elif case["op"] == "linear_bwd":
        s["dy"] = randn(case["m"], case["n"]).to(torch.bfloat16)
        s["z"] = (2.0 * randn(case["m"], case["n"])).to(torch.bfloat16)
    else:
        m, h = case["m"], case["h"]
        x = _acts(gen, m, h) + 0.25
        s["x"] = x.to(_TYPES[case["x"]])
        s["w"] = (1.0 + 0.1 * randn(h)).to(_TYPES[case["w"]])
        if case["op"] == "norm":
            s["b"] = (0.1 * randn(h)).to(_TYPES[case["w"]])
            s["sy"] = torch.full((1,), 16.0 / 448.0, device="cuda") if case["out"] == "fp8" else None
        else:
            s["dy"] = randn(m, h).to(_TYPES[case["dy"]])
            s["dres"] = randn(m, h).to(_TYPES[case["x"]]) if case["dres"] else None
            # what the forward pass kept
            d = s["x"].double()
            mean = d.mean(dim=1)
            var = (d - mean[:, None]).square().mean(dim=1)
            s["mean"], s["rstd"] = mean.float(), (1.0 / torch.sqrt(var + EPS)).float()
    return s


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    import mlp_fp8_quant_amd as fw

    case = s["case"]
    outs = {"bf16": fw.OUT_BF16, "fp8": fw.OUT_FP8, "f32": fw.OUT_F32}
    acts = {"none": fw.ACT_NONE, "relu": fw.ACT_RELU, "gelu": fw.ACT_GELU,
            "gelu_tanh": fw.ACT_GELU_TANH, "silu": fw.ACT_SILU}
    values = lambda y: y.view(torch.float8_e4m3fn) if y.dtype == torch.uint8 else y  # noqa: E731
    if case["op"] == "linear":
        r = fw.fp8_linear_act(s["qx"], s["qw"], s["sx"], s["sw"], bias=s["bias"], act=acts[case["act"]],
                              residual=s["residual"], out_kind=outs[case["out"]], sy=s["sy"],
                              rowwise=case["rowwise"], pre=case["pre"])
        return (values(r[0]), r[1]) if case["pre"] else values(r)
    if case["op"] == "linear_bwd":
        return fw.fp8_linear_act_backward(s["dy"], s["z"], act=acts[case["act"]])
    if case["op"] == "norm":
        r = fw.fp8_layer_norm(s["x"], s["w"], s["b"], eps=EPS, out_kind=outs[case["out"]], sy=s["sy"],
                              stats=case["stats"])
        return (values(r[0]), r[1], r[2]) if case["stats"] else values(r)
    return fw.fp8_layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], dres=s["dres"])


# ---------------------------------------------------------------------------
# The plain form, in 32 bits
# ---------------------------------------------------------------------------

_SQRT_2_OVER_PI = math.sqrt(2.0 / math.pi)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(_SQRT_2_OVER_PI * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(_SQRT_2_OVER_PI * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _SQRT_2_OVER_PI * (1.0 + 3.0 * 0.044715 * z * z)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _emit(y, out, sy):
    if out == "fp8":
        return (y / sy).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return y.to(_TYPES[out])


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    if case["op"] == "linear":
        acc = s["qx"].view(torch.float8_e4m3fn).float() @ s["qw"].view(torch.float8_e4m3fn).float().t()
        z = acc * (s["sx"][:, None] * s["sw"][None, :] if case["rowwise"] else s["sx"] * s["sw"])
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        y = _emit(y, case["out"], s["sy"])
        return (y, z.to(torch.bfloat16)) if case["pre"] else y
    if case["op"] == "linear_bwd":
        dz = s["dy"].float() * _act_slope(s["z"].float(), case["act"])
        return dz.to(torch.bfloat16), dz.sum(dim=0)
    x = s["x"].float()
    if case["op"] == "norm":
        mean = x.mean(dim=1)
        xc = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((xc * xc).mean(dim=1) + EPS)
        y = _emit(xc * rstd[:, None] * s["w"].float() + s["b"].float(), case["out"], s["sy"])
        return (y, mean, rstd) if case["stats"] else y
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    g = dy * s["w"].float()
    dx = rstd * (g - g.mean(dim=1, keepdim=True) - xh * (g * xh).mean(dim=1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dx.to(s["x"].dtype), (dy * xh).sum(dim=0), dy.sum(dim=0)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

_SIZE = {"none": 0, "fp8": 1, "bf16": 2, "f32": 4}


def work(case):
    m = case["m"]
    if case["op"] == "linear":
        n, k = case["n"], case["k"]
        per = _SIZE[case["residual"]] + _SIZE[case["out"]] + (2 if case["pre"] else 0)
        scales = 4 * (m + n) if case["rowwise"] else 8
        return {"bytes": m * k + n * k + m * n * per + n * _SIZE[case["bias"]] + scales, "flops": 2 * m * n * k}
    if case["op"] == "linear_bwd":
        n = case["n"]
        return {"bytes": 6 * m * n + 4 * n, "flops": 12 * m * n}
    h = case["h"]
    if case["op"] == "norm":
        return {"bytes": m * h * (_SIZE[case["x"]] + _SIZE[case["out"]]) + 2 * h * _SIZE[case["w"]]
                + (8 * m if case["stats"] else 0), "flops": 8 * m * h}
    per = 2 * _SIZE[case["x"]] + _SIZE[case["dy"]] + (_SIZE[case["x"]] if case["dres"] else 0)
    return {"bytes": m * h * per + h * (_SIZE[case["w"]] + 8) + 8 * m, "flops": 16 * m * h}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _decode(q):
    """Values of E4M3 codes from their fields: (-1)^s 2^(e-7) (1 + f/8), or 2^-6 f/8 where e is 0."""
    u = q.to(torch.int32)
    e, f = (u >> 3) & 15, (u & 7).double() / 8.0
    v = torch.where(e == 0, f * 2.0 ** -6, torch.ldexp(1.0 + f, (e - 7).double()))
    return torch.where(u >= 128, -v, v)


def _phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def exact(case, seed):
    s = prepare(case, seed)
    act = case.get("act")
    wide = lambda t: t.to(torch.float64)  # noqa: E731
    if case["op"] == "linear":
        z = torch.mm(_decode(s["qx"]), _decode(s["qw"]).t().contiguous())
        # the scale of a product is one 32-bit number by the operator's definition
        z *= wide(torch.outer(s["sx"], s["sw"]))
        if s["bias"] is not None:
            z += wide(s["bias"])
        if act == "relu":
            y = z.clamp(min=0.0)
        elif act == "gelu":
            y = z * _phi(z)
        elif act == "gelu_tanh":
            y = z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
        elif act == "silu":
            y = z * torch.sigmoid(z)
        else:
            y = z.clone()
        if s["residual"] is not None:
            y += wide(s["residual"])
        if case["out"] == "fp8":
            y = (y / wide(s["sy"])).clamp(-448.0, 448.0)
        return (y, z) if case["pre"] else y
    if case["op"] == "linear_bwd":
        z = wide(s["z"])
        if act == "relu":
            d = torch.where(z > 0, 1.0, 0.0)
        elif act == "gelu":
            d = _phi(z) + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
        elif act == "gelu_tanh":
            c = math.sqrt(2.0 / math.pi)
            p = torch.sigmoid(2.0 * c * (z + 0.044715 * z ** 3))
            d = p + 2.0 * c * z * p * (1.0 - p) * (1.0 + 0.134145 * z ** 2)
        elif act == "silu":
            p = torch.sigmoid(z)
            d = p + z * p * (1.0 - p)
        else:
            d = torch.ones_like(z)
        d = d * wide(s["dy"])
        return d, d.sum(dim=0)
    x, w = wide(s["x"]), wide(s["w"])
    if case["op"] == "norm":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        r = torch.rsqrt(var + EPS)
        y = torch.addcmul(wide(s["b"]), (x - mean[:, None]) * r[:, None], w)
        if case["out"] == "fp8":
            y = (y / wide(s["sy"])).clamp(-448.0, 448.0)
        return (y, mean, r) if case["stats"] else y
    dy, r = wide(s["dy"]), wide(s["rstd"])[:, None]
    xh = (x - wide(s["mean"])[:, None]) * r
    g = dy * w
    h = x.shape[1]
    dx = r / h * (h * g - g.sum(1, keepdim=True) - xh * torch.sum(g * xh, 1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + wide(s["dres"])
    return dx, torch.sum(dy * xh, 0), torch.sum(dy, 0)
