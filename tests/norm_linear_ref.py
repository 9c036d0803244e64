"""Plain 64-bit references of the Linear epilogue and the layer norm with
their backward passes (torch on the CPU, from the formulas), and the error
bounds that the GPU tests hold the kernels to.

u = 2^-24 is half a step of FP32 relative to the value.  The bounds count the
kernels' roundings; each is spelled out at its function.  An output's own
rounding adds half a step of its type: 2^-8 of the value for BF16, 2^-4 for
E4M3 (2^-10 below its smallest normal).
"""

import math

import torch

U = 2.0 ** -24
BF16_HALF, E4M3_HALF, E4M3_SUB_HALF, E4M3_MAX = 2.0 ** -8, 2.0 ** -4, 2.0 ** -10, 448.0
NONE, RELU, GELU, GELU_TANH, SILU = range(5)
ACTS = (NONE, RELU, GELU, GELU_TANH, SILU)
_C = math.sqrt(2.0 / math.pi)


def decode(q):
    """Values of E4M3 codes, float64 (0x7F and 0xFF are NaN)."""
    return q.cpu().view(torch.float8_e4m3fn).double()


def phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def tanh_arg(z):
    return 2.0 * _C * (z + 0.044715 * z ** 3)


def act(z, kind):
    if kind == RELU:
        return torch.where(z > 0, z, torch.zeros_like(z))
    if kind == GELU:
        return z * phi(z)
    if kind == GELU_TANH:
        return z * torch.sigmoid(tanh_arg(z))
    if kind == SILU:
        return z * torch.sigmoid(z)
    return z.clone()


def act_slope(z, kind):
    if kind == RELU:
        return (z > 0).double()
    if kind == GELU:
        return phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == GELU_TANH:
        p = torch.sigmoid(tanh_arg(z))
        return p + z * p * (1 - p) * 2 * _C * (1 + 3 * 0.044715 * z * z)
    if kind == SILU:
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def act_error(z, kind):
    """Bound of the kernel's own error in act(z).

    sigma(x): the exponential's argument x log2(e) rounds to u |x| absolute
    (and the constant to u |x|), the exponential and the reciprocal take a
    step (2 u) each, the sum u, the product with z u: (2 |x| + 6) u.
    gelu_tanh's argument adds five roundings, 5 |x| u.  gelu: formula 7.1.26
    of Abramowitz and Stegun is within 1.5e-7 for erfc, half that for Phi; its
    evaluation takes about 16 roundings and the exponential's argument z^2/2,
    rounded four times, 2 z^2 u, relative to a value of at most
    exp(-z^2/2) / 2 <= 1/2.
    """
    a = z.abs()
    if kind in (NONE, RELU):
        return torch.zeros_like(a)
    if kind == SILU:
        return act(z, kind).abs() * (2 * a + 6) * U
    if kind == GELU_TANH:
        return act(z, kind).abs() * (7 * tanh_arg(a) + 6) * U
    tail = torch.exp(-z * z / 2) / 2
    return a * (0.75e-7 + (16 + 2 * z * z) * U * tail + 2 * U)


def act_slope_error(z, kind):
    """Bound of the kernel's error in act'(z), from the errors of sigma and
    Phi above: |z| times the one in sigma (1 - sigma) next to sigma's own."""
    a = z.abs()
    if kind in (NONE, RELU):
        return torch.zeros_like(a)
    if kind == SILU:
        return (2 * a + 8) * U * (1 + a)
    if kind == GELU_TANH:
        x = tanh_arg(a.clamp(max=6.0))       # beyond 6 sigma is 0 or 1 to 1e-16
        return (7 * x + 10) * U * (1 + a.clamp(max=6.0) * 2 * _C * (1 + 3 * 0.044715 * a.clamp(max=6.0) ** 2))
    tail = torch.exp(-z * z / 2)
    return 0.75e-7 + (20 + 4 * z * z) * U * tail * (1 + a) + 2 * U


def linear_act(qx, qw, sx, sw, bias, kind, residual):
    """(y, z, err, err_z) in float64 with err the bound of the kernel's error
    before the output's rounding.

    The products are exact; the sum is held to the library's GEMM bar,
    1e-5 alpha sum|terms| (K/16 MFMA additions and the join of the partial sums,
    each half a step of at most sum|terms|: (K/16 + 16) u stays below it up
    to K = 2400).  alpha, alpha acc, the bias's and the residual's addition
    round once each; act's slope is below 1.13.
    """
    a, b = decode(qx), decode(qw)
    alpha = (sx.cpu().float().reshape(-1, 1) * sw.cpu().float().reshape(1, -1)).double()
    s = a @ b.t()
    terms = a.abs() @ b.abs().t()
    z = s * alpha
    err_z = 1e-5 * alpha.abs() * terms + z.abs() * U
    if bias is not None:
        z = z + bias.cpu().double()
    err_z = err_z + z.abs() * U
    y = act(z, kind)
    err = 1.13 * err_z + act_error(z, kind)
    if residual is not None:
        y = y + residual.cpu().double()
        err = err + y.abs() * U
    return y, z, err, err_z


def norm(x, w, b, eps):
    """(y, mean, rstd, err) of the layer norm; err as in norm_errors."""
    x = x.cpu().double()
    mean = x.mean(dim=-1)
    var = (x - mean[..., None]).square().mean(dim=-1)
    rstd = 1.0 / torch.sqrt(var + eps)
    xh = (x - mean[..., None]) * rstd[..., None]
    y = xh if w is None else xh * w.cpu().double()
    e_mean, e_rstd = norm_errors(x, eps)
    err = y.abs() * (e_rstd[..., None] + 4 * U) + \
        (e_mean * rstd)[..., None] * (1.0 if w is None else w.cpu().double().abs())
    if b is not None:
        y = y + b.cpu().double()
    err = err + y.abs() * U
    return y, mean, rstd, err


def norm_errors(x, eps):
    """Bounds (mean absolute, rstd relative).  A sum of H values takes at most
    H/64 + 16 additions one after another (64 lanes or more side by side, then
    a tree), each half a step of at most sum|x|; the product with 1/H two
    more.  The variance about a mean off by e is off by e^2 (the differences
    sum to zero), beside such a sum's relative error and the rounding and
    squaring of each difference."""
    H = x.shape[-1]
    d = (H / 64 + 18) * U
    mean = x.mean(dim=-1)
    e_mean = d * x.abs().mean(dim=-1)
    var = (x - mean[..., None]).square().mean(dim=-1)
    e_var = (var + e_mean ** 2) * (d + 4 * U) + e_mean ** 2
    e_rstd = 0.5 * e_var / (var + eps) + 4 * U
    return e_mean, e_rstd


def norm_backward(dy, x, w, mean, rstd, dres):
    """(dx, dw, db, err_dx, err_dw, err_db) for given FP32 mean and rstd.

    Sums over a row as in norm_errors; sums over rows take at most rows + 16
    additions one after another.  xh rounds twice (u |xh| each; the difference
    relative to itself), g once, the combination four times.
    """
    dy, x = dy.cpu().double(), x.cpu().double()
    mean, rstd = mean.cpu().double()[..., None], rstd.cpu().double()[..., None]
    H = x.shape[-1]
    rows = x.numel() // max(H, 1)
    xh = (x - mean) * rstd
    g = dy if w is None else dy * w.cpu().double()
    c1 = g.mean(dim=-1, keepdim=True)
    c2 = (g * xh).mean(dim=-1, keepdim=True)
    dx = rstd * (g - c1 - xh * c2)
    d = (H / 64 + 20) * U
    e1 = d * g.abs().mean(dim=-1, keepdim=True)
    e2 = d * (g * xh).abs().mean(dim=-1, keepdim=True)
    err_dx = rstd * (g.abs() * 4 * U + c1.abs() * 4 * U + (xh * c2).abs() * 6 * U + e1 + xh.abs() * e2) \
        + dx.abs() * 2 * U
    if dres is not None:
        dx = dx + dres.cpu().double()
        err_dx = err_dx + dx.abs() * U
    flat = lambda t: t.reshape(-1, H)  # noqa: E731
    dr = (rows + 20) * U
    dw, db = flat(dy * xh).sum(0), flat(dy).sum(0)
    return (dx, dw, db, err_dx, dr * flat(dy * xh).abs().sum(0), dr * flat(dy).abs().sum(0))


def check(got, want, err, what=""):
    """A BF16 or FP32 output within err and its own rounding; NaN and
    infinities where the reference has them."""
    got64 = got.cpu().double().reshape(want.shape)
    half = BF16_HALF if got.dtype == torch.bfloat16 else U
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got64), torch.isnan(want)), f"{what}: NaN elsewhere"
    inf = ~fine & ~torch.isnan(want)
    assert torch.equal(got64[inf], want[inf]), f"{what}: infinities"
    off = (got64 - want).abs()[fine]
    tol = (err + (want.abs() + err) * half)[fine] + 2.0 ** -140
    worst = (off / tol).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {int((off > tol).sum())} of {off.numel()} outside, worst {worst:.3g} of the bound"
    return worst


def check_fp8(codes, want, err, sy, what=""):
    """E4M3 codes of want / sy, saturated at 448 (an infinity too; NaN is a
    NaN code)."""
    s = sy.cpu().double()
    got = decode(codes).reshape(want.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN elsewhere"
    fine = ~torch.isnan(want)
    t = (want / s)
    # 1 / sy and the product with it round once each, and their product's error term a third
    e = (torch.where(torch.isfinite(err), err, torch.zeros_like(err)) / s) + t.abs().clamp(max=1e30) * 3 * U
    t = t.clamp(-E4M3_MAX, E4M3_MAX)
    off = (got - t).abs()[fine]
    tol = (e + torch.maximum((t.abs() + e) * E4M3_HALF, torch.full_like(t, E4M3_SUB_HALF)))[fine]
    worst = (off / tol).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {int((off > tol).sum())} codes outside, worst {worst:.3g}"
