"""Block-scaled FP8 products and the residual stream's norms as measured workloads.

Five operators: quantization of a tensor with an FP32 scale for each block of
128 (along rows, along columns, or 128 x 128), SwiGLU that emits such codes,
the product of two block-scaled operands with bias, activation and residual,
and the norms before and after a block fused with the block's gate and
residual scale, forward and backward.  ``run`` computes a case in plain torch
operations in 32 bits, or, with ``own`` true, through ``mlp_fp8_quant_amd``;
``exact`` is the definition in 64 bits.  FP8 results are returned as float8
values beside their scales.
"""

import math

import torch

own = False

EPS = 1e-6
BLOCK = 128
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _quant(name, m, k, x, tile, transpose):
    return {"name": name, "op": "quant", "m": m, "k": k, "x": x, "tile": tile, "transpose": transpose}


def _silu(name, m, k):
    return {"name": name, "op": "silu", "m": m, "k": k}


def _linear(name, m, n, k, ws, bias, act, residual, out):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "ws": ws, "bias": bias, "act": act,
            "residual": residual, "out": out}


def _norm(name, m, h, x, hid, w, post, gates, alpha, out, stats):
    return {"name": name, "op": "norm", "m": m, "h": h, "x": x, "hid": hid, "w": w, "post": post,
            "gates": gates, "alpha": alpha, "out": out, "stats": stats}


def _norm_bwd(name, m, h, x, hid, w, post, gates, alpha, dr):
    return {"name": name, "op": "norm_bwd", "m": m, "h": h, "x": x, "hid": hid, "w": w, "post": post,
            "gates": gates, "alpha": alpha, "dr": dr}


def listed():
    return [
        # the gradient of a ragged batch, quantized along its tokens for the weight's gradient
        _quant("quant ragged transposed", 1531, 2053, "bf16", False, True),
        # the large tower's up projection quantized at load, a scale for each 128 x 128 tile
        _quant("quant large weight", 25600, 5120, "bf16", True, False),
        # SwiGLU of a few decoded tokens, codes for the down projection
        _silu("silu 13 tokens", 13, 12288),
        # SwiGLU of the generation tower's batch
        _silu("silu gen", 4096, 12288),
        # one token through the decoder layer's o projection, added to the residual stream
        _linear("linear token o", 1, 4096, 4096, "tile", "none", "none", "bf16", "bf16"),
        # the understanding tower's down projection (512 tokens) with its residual
        _linear("linear 512 tokens down", 512, 4096, 12288, "tile", "none", "none", "bf16", "bf16"),
        # a weight's gradient at sizes no tile divides, summed over 1531 tokens onto the gradient so far
        _linear("linear ragged weight gradient", 2053, 1027, 1531, "row", "none", "none", "f32", "f32"),
        # the large tower's up projection
        _linear("linear large up", 16384, 25600, 5120, "tile", "bf16", "none", "none", "bf16"),
        # one token between two blocks: post-norm, gate, residual, pre-norm, codes
        _norm("norm token", 1, 4096, "bf16", "bf16", "bf16", True, 1, 1.0, "block", False),
        # the large tower's batch of 8 samples, each with a gate of its own
        _norm("norm large", 16384, 5120, "bf16", "bf16", "bf16", True, 8, 1.0, "block", False),
        # backward at the understanding tower's size, and at the large tower's with the stream's gradient
        _norm_bwd("norm backward 512 tokens", 512, 4096, "bf16", "bf16", "f32", True, 1, 0.5, False),
        _norm_bwd("norm backward large", 16384, 5120, "bf16", "bf16", "bf16", True, 8, 1.0, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _gated(rng):
    """Rows, and how many gates they share (none, one, or one for each sample of equal length)."""
    gates = rng.choice([0, 1, _log(rng, 2, 64)])
    return max(1, gates) * _log(rng, 1, max(1, 12000 // max(1, gates))), gates


def draw(rng):
    op = rng.choice(["quant", "silu", "linear", "linear", "norm", "norm_bwd"])
    if op == "quant":
        c = _quant("", _log(rng, 1, 12000), _log(rng, 16, 12288), rng.choice(["bf16", "bf16", "f32"]),
                   rng.random() < 0.3, rng.random() < 0.5)
    elif op == "silu":
        c = _silu("", _log(rng, 1, 12000), _log(rng, 64, 12288))
    elif op == "linear":
        c = _linear("", _log(rng, 1, 6000), _log(rng, 64, 16384), _log(rng, 64, 12288),
                    rng.choice(["tile", "tile", "row"]), rng.choice(["none", "bf16", "f32"]),
                    rng.choice(["none", "none", "gelu_tanh", "silu"]), rng.choice(["none", "bf16", "f32"]),
                    rng.choice(["bf16", "bf16", "f32"]))
    else:
        m, gates = _gated(rng)
        h, x, hid = _log(rng, 32, 8192), rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "bf16", "f32"])
        w, post, alpha = rng.choice(["bf16", "f32"]), rng.random() < 0.5, rng.choice([1.0, 0.22])
        if op == "norm":
            c = _norm("", m, h, x, hid, w, post, gates, alpha, rng.choice(["bf16", "block", "fp8", "f32"]),
                      rng.random() < 0.5)
        else:
            c = _norm_bwd("", m, h, x, hid, w, post, gates, alpha, rng.random() < 0.7)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _up(n, to):
    return (n + to - 1) // to * to


def _acts(gen, rows, cols):
    """N(0, 1) with 0.5% of the entries times 20; the last rows of a batch are its padding, zero."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x = torch.where(torch.rand(rows, cols, generator=gen, device="cuda") < 0.005, 20.0 * x, x)
    if rows >= 64:
        x[rows - rows // 64:] = 0.0
    return x


def _spread(s, tile, rows, k):
    """The scale of every element of [rows, k] from one per group of 128 (or per 128 x 128 tile)."""
    s = s.repeat_interleave(BLOCK, dim=1)[:, :k]
    return s.repeat_interleave(BLOCK, dim=0)[:rows] if tile else s


def _block_codes(x, tile, pad=True):
    """(codes as values, scales) of x [rows, k]: scale amax / 448 of each group of 128 of a row, or of each
    128 x 128 tile; rows of codes filled up with zeros to a multiple of 16."""
    rows, k = x.shape
    kb = _up(k, BLOCK)
    f = torch.nn.functional.pad(x, (0, kb - k, 0, _up(rows, BLOCK) - rows if tile else 0))
    a = f.abs().view(-1, BLOCK if tile else 1, kb // BLOCK, BLOCK).amax(dim=(1, 3))
    s = a / 448.0
    e = _spread(s, tile, rows, k)
    q = torch.where(e > 0, x / torch.where(e > 0, e, torch.ones_like(e)), x).clamp(-448.0, 448.0)
    if pad:
        q = torch.nn.functional.pad(q, (0, _up(k, 16) - k))
    return q.to(torch.float8_e4m3fn), s


def _weights(randn, *shape, like):
    return (1.0 + 0.1 * randn(*shape)).to(_TYPES[like])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    s = {"case": case}
    m = case["m"]
    if case["op"] == "quant":
        x = 0.02 * randn(m, case["k"]) if case["tile"] else _acts(gen, m, case["k"])
        s["x"] = x.to(_TYPES[case["x"]])
    elif case["op"] == "silu":
        s["g"] = (2.0 * randn(m, case["k"])).to(torch.bfloat16)
        s["u"] = _acts(gen, m, case["k"]).to(torch.bfloat16)
    elif case["op"] == "linear":
        n, k = case["n"], case["k"]
        tile = case["ws"] == "tile"
        qx, s["sx"] = _block_codes(_acts(gen, m, k).to(torch.bfloat16).float(), False)
        # a weight, or (a scale for each row) the other operand of a weight's gradient
        w = 0.02 * randn(n, k) if tile else _acts(gen, n, k)
        qw, s["sw"] = _block_codes(w.to(torch.bfloat16).float(), tile)
        s["qx"], s["qw"] = qx.view(torch.uint8), qw.view(torch.uint8)
        s["bias"] = None if case["bias"] == "none" else (0.1 * randn(n)).to(_TYPES[case["bias"]])
        s["residual"] = None if case["residual"] == "none" else _acts(gen, m, n).to(_TYPES[case["residual"]])
    else:
        h = case["h"]
        x, hid = _acts(gen, m, h), 0.7 * _acts(gen, m, h)
        s["hid"] = hid.to(_TYPES[case["hid"]])
        s["w"] = _weights(randn, h, like=case["w"])
        s["post"] = _weights(randn, h, like=case["w"]) if case["post"] else None
        s["gate"] = (0.5 + 0.3 * randn(case["gates"], h)).to(_TYPES[case["w"]]) if case["gates"] else None
        if case["op"] == "norm":
            s["x"] = x.to(_TYPES[case["x"]])
            s["sy"] = torch.full((1,), 16.0 / 448.0, device="cuda") if case["out"] == "fp8" else None
        else:
            # the stream after the block, what the forward pass kept, and the gradients that arrive
            s["r"] = (x + hid).to(_TYPES[case["x"]])
            keep = lambda t: (1.0 / torch.sqrt(t.double().square().mean(dim=1) + EPS)).float()  # noqa: E731
            s["rstd"], s["post_rstd"] = keep(s["r"]), keep(s["hid"]) if case["post"] else None
            s["dy"] = randn(m, h).to(_TYPES[case["hid"]])
            s["dr"] = randn(m, h).to(_TYPES[case["x"]]) if case["dr"] else None
    return s


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    import mlp_fp8_quant_amd as fw

    case = s["case"]
    outs = {"bf16": fw.OUT_BF16, "fp8": fw.OUT_FP8, "f32": fw.OUT_F32, "block": fw.OUT_FP8_BLOCK}
    acts = {"none": fw.ACT_NONE, "gelu_tanh": fw.ACT_GELU_TANH, "silu": fw.ACT_SILU}
    values = lambda y: y.view(torch.float8_e4m3fn) if y.dtype == torch.uint8 else y  # noqa: E731
    if case["op"] == "quant":
        q, sc = fw.fp8_quant_block(s["x"], tile=case["tile"], transpose=case["transpose"])
        return values(q), sc
    if case["op"] == "silu":
        q, sc = fw.silu_mul_2in_block(s["g"], s["u"])
        return values(q), sc
    if case["op"] == "linear":
        return fw.fp8_linear_block(s["qx"], s["qw"], s["sx"], s["sw"], bias=s["bias"], act=acts[case["act"]],
                                   residual=s["residual"], out_kind=outs[case["out"]])
    if case["op"] == "norm":
        r = fw.fp8_residual_norm(s["x"], s["w"], s["hid"], gate=s["gate"], post_weight=s["post"],
                                 alpha=case["alpha"], eps=EPS, out_kind=outs[case["out"]], sy=s["sy"],
                                 stats=case["stats"])
        y = (values(r[0][0]), r[0][1]) if case["out"] == "block" else (values(r[0]),)
        return y + tuple(t for t in r[1:] if t is not None)
    r = fw.fp8_residual_norm_backward(s["dy"], s["r"], s["w"], s["rstd"], s["hid"], gate=s["gate"],
                                      post_weight=s["post"], post_rstd=s["post_rstd"], alpha=case["alpha"],
                                      dr=s["dr"])
    return tuple(t for t in r if t is not None)


# ---------------------------------------------------------------------------
# The plain form, in 32 bits
# ---------------------------------------------------------------------------

def _act(z, act):
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _rows_of(gate, m):
    return gate.float().repeat_interleave(m // gate.shape[0], dim=0)


def _run_norm(s, case):
    x, v, m = s["x"].float(), s["hid"].float(), case["m"]
    post_rstd = None
    if s["post"] is not None:
        post_rstd = 1.0 / torch.sqrt((v * v).mean(dim=1) + EPS)
        v = v * post_rstd[:, None] * s["post"].float()
    if s["gate"] is not None:
        v = v * _rows_of(s["gate"], m)
    r = x + case["alpha"] * v
    rstd = 1.0 / torch.sqrt((r * r).mean(dim=1) + EPS)
    y = r * rstd[:, None] * s["w"].float()
    if case["out"] == "block":
        y = _block_codes(y, False)
    elif case["out"] == "fp8":
        y = ((y / s["sy"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn),)
    else:
        y = (y.to(_TYPES[case["out"]]),)
    y = y + (r.to(s["x"].dtype),)
    if case["stats"]:
        y = y + (rstd,) + (() if post_rstd is None else (post_rstd,))
    return y


def _run_norm_bwd(s, case):
    m, h = case["m"], case["h"]
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    rh = s["r"].float() * rstd
    g = dy * s["w"].float()
    dx = rstd * (g - rh * (g * rh).mean(dim=1, keepdim=True))
    if s["dr"] is not None:
        dx = dx + s["dr"].float()
    hh = s["hid"].float()
    if s["post"] is not None:
        hh = hh * s["post_rstd"][:, None]
    dv = case["alpha"] * dx
    a = dv * hh                                        # the gate's gradient before the post-norm's weight
    gate = None if s["gate"] is None else _rows_of(s["gate"], m)
    if gate is not None:
        dv = dv * gate
    outs = (dx.to(s["r"].dtype),)
    if s["post"] is not None:
        p = dv * s["post"].float()
        dh = s["post_rstd"][:, None] * (p - hh * (p * hh).mean(dim=1, keepdim=True))
    else:
        dh = dv
    outs += (dh.to(s["hid"].dtype), (dy * rh).sum(dim=0))
    if gate is not None:
        ga = a if s["post"] is None else a * s["post"].float()
        outs += (ga.view(case["gates"], m // case["gates"], h).sum(dim=1),)
    if s["post"] is not None:
        outs += ((dv * hh).sum(dim=0),)
    return outs


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    if case["op"] == "quant":
        x = s["x"].float()
        return _block_codes(x.t().contiguous() if case["transpose"] else x, case["tile"])
    if case["op"] == "silu":
        g = s["g"].float()
        return _block_codes(g / (1.0 + torch.exp(-g)) * s["u"].float(), False)
    if case["op"] == "linear":
        m, n = case["m"], case["n"]
        kp = s["qx"].shape[1]
        x = s["qx"].view(torch.float8_e4m3fn).float() * _spread(s["sx"], False, m, kp)
        w = s["qw"].view(torch.float8_e4m3fn).float() * _spread(s["sw"], case["ws"] == "tile", n, kp)
        z = x @ w.t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(_TYPES[case["out"]])
    return _run_norm(s, case) if case["op"] == "norm" else _run_norm_bwd(s, case)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

_SIZE = {"none": 0, "fp8": 1, "bf16": 2, "f32": 4}


def work(case):
    m = case["m"]
    blocks = lambda n: (n + BLOCK - 1) // BLOCK  # noqa: E731
    if case["op"] in ("quant", "silu"):
        k = case["k"]
        rows, cols = (k, m) if case.get("transpose") else (m, k)
        scales = blocks(rows) * blocks(cols) if case.get("tile") else rows * blocks(cols)
        each = _SIZE[case["x"]] if case["op"] == "quant" else 4
        return {"bytes": m * k * each + rows * _up(cols, 16) + 4 * scales,
                "flops": m * k * (3 if case["op"] == "quant" else 8)}
    if case["op"] == "linear":
        n, k = case["n"], case["k"]
        kb = blocks(k)
        scales = m * kb + (blocks(n) if case["ws"] == "tile" else n) * kb
        return {"bytes": (m + n) * _up(k, 16) + m * n * (_SIZE[case["residual"]] + _SIZE[case["out"]])
                + n * _SIZE[case["bias"]] + 4 * scales, "flops": 2 * m * n * k}
    h, gates = case["h"], case["gates"]
    small = h * _SIZE[case["w"]] * (1 + (1 if case["post"] else 0) + gates)
    if case["op"] == "norm":
        out = 1 + 4 / BLOCK if case["out"] == "block" else _SIZE[case["out"]]
        stats = 4 * m * (2 if case["post"] else 1) if case["stats"] else 0
        return {"bytes": round(m * h * (2 * _SIZE[case["x"]] + _SIZE[case["hid"]] + out)) + small + stats,
                "flops": m * h * (12 if case["post"] else 8)}
    per = (2 + (1 if case["dr"] else 0)) * _SIZE[case["x"]] + 3 * _SIZE[case["hid"]]
    sums = 4 * h * (1 + (1 if case["post"] else 0) + gates)
    return {"bytes": m * h * per + small + sums + 4 * m * (2 if case["post"] else 1),
            "flops": m * h * (24 if case["post"] else 14)}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _decode(q):
    """Values of E4M3 codes from their fields: (-1)^s 2^(e-7) (1 + f/8), or 2^-6 f/8 where e is 0."""
    u = q.to(torch.int32)
    e, f = (u >> 3) & 15, (u & 7).double() / 8.0
    v = torch.where(e == 0, f * 2.0 ** -6, torch.ldexp(1.0 + f, (e - 7).double()))
    return torch.where(u >= 128, -v, v)


def _scaled(x, tile):
    """[x / scale with zeros up to a multiple of 16 columns, scale] in 64 bits, block by block of columns."""
    rows, k = x.shape
    q = torch.zeros(rows, _up(k, 16), dtype=torch.float64, device=x.device)
    scales = []
    for c in range(0, k, BLOCK):
        b = x[:, c:c + BLOCK]
        top = b.abs().max(dim=1).values
        if tile:
            top = torch.stack([t.max() for t in top.split(BLOCK)])
        scales.append(top / 448.0)
        d = scales[-1].repeat_interleave(BLOCK)[:rows] if tile else scales[-1]
        q[:, c:c + b.shape[1]] = torch.nan_to_num(b / d[:, None], nan=0.0)
    return q, torch.stack(scales, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    wide = lambda t: t.to(torch.float64)  # noqa: E731
    if case["op"] == "quant":
        x = wide(s["x"])
        return _scaled(x.t() if case["transpose"] else x, case["tile"])
    if case["op"] == "silu":
        return _scaled(wide(s["g"]) * torch.sigmoid(wide(s["g"])) * wide(s["u"]), False)
    if case["op"] == "linear":
        m, n = case["m"], case["n"]
        x, w = _decode(s["qx"]), _decode(s["qw"])
        for b in range(s["sx"].shape[1]):
            c = slice(b * BLOCK, (b + 1) * BLOCK)
            x[:, c] *= wide(s["sx"])[:, b:b + 1]
            col = wide(s["sw"])[:, b]
            w[:, c] *= (col.repeat_interleave(BLOCK)[:n] if case["ws"] == "tile" else col)[:, None]
        z = torch.mm(x, w.t())
        if s["bias"] is not None:
            z += wide(s["bias"])
        if case["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif case["act"] == "gelu_tanh":
            z = z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
        if s["residual"] is not None:
            z += wide(s["residual"])
        return z
    m, h = case["m"], case["h"]
    hid, w = wide(s["hid"]), wide(s["w"])
    each = torch.arange(m, device="cuda") // (m // case["gates"]) if case["gates"] else None
    gate = 1.0 if each is None else wide(s["gate"])[each]
    if case["op"] == "norm":
        t = hid.square().sum(dim=1).div(h).add(EPS).rsqrt()
        v = hid * t[:, None] * wide(s["post"]) if case["post"] else hid
        r = wide(s["x"]) + case["alpha"] * gate * v
        q = r.square().sum(dim=1).div(h).add(EPS).rsqrt()
        y = r * q[:, None] * w
        if case["out"] == "block":
            y = _scaled(y, False)
        elif case["out"] == "fp8":
            y = ((y / wide(s["sy"])).clamp(-448.0, 448.0),)
        else:
            y = (y,)
        return y + (r,) + ((q,) + ((t,) if case["post"] else ()) if case["stats"] else ())
    dy, q = wide(s["dy"]), wide(s["rstd"])[:, None]
    n = wide(s["r"]) * q
    dx = q * (dy * w - n * torch.sum(dy * w * n, 1, keepdim=True) / h)
    if s["dr"] is not None:
        dx = dx + wide(s["dr"])
    z = hid * wide(s["post_rstd"])[:, None] if case["post"] else hid
    b = wide(s["post"]) if case["post"] else 1.0
    d = case["alpha"] * gate * b * dx
    dh = wide(s["post_rstd"])[:, None] * (d - z * torch.sum(d * z, 1, keepdim=True) / h) if case["post"] else d
    outs = (dx, dh, torch.sum(dy * n, 0))
    if each is not None:
        into = torch.zeros(case["gates"], h, dtype=torch.float64, device="cuda")
        outs += (into.index_add_(0, each, case["alpha"] * b * z * dx),)
    if case["post"]:
        outs += (torch.sum(case["alpha"] * gate * z * dx, 0),)
    return outs
