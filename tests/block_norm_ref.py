"""Plain references of the block-scaled FP8 calls and of the residual stream's
norms with their backward pass (torch and NumPy on the CPU, from the formulas),
and the error bounds that the GPU tests hold the kernels to.

u = 2^-24 is half a step of FP32 relative to the value; the bounds count the
kernels' roundings, spelled out at each function.
"""

import numpy as np
import torch

from norm_linear_ref import E4M3_HALF, E4M3_SUB_HALF, U, act, act_error, check, decode  # noqa: F401
from oracle.formats import e4m3_encode

BLOCK = 128


def up(n, to):
    return (n + to - 1) // to * to


def spread(s, tile, rows, cols):
    """Every element's scale from one per 128 columns of a row, or per 128 x 128 tile."""
    s = s.repeat_interleave(BLOCK, dim=1)[:, :cols]
    return s.repeat_interleave(BLOCK, dim=0)[:rows] if tile else s


def block_amax(x, tile):
    rows, cols = x.shape
    f = torch.nn.functional.pad(x.abs(), (0, up(cols, BLOCK) - cols, 0, up(rows, BLOCK) - rows if tile else 0))
    return f.view(-1, BLOCK if tile else 1, f.shape[1] // BLOCK, BLOCK).amax(dim=(1, 3))


def quant(x, tile, transpose):
    """(codes, scales) of x [M, K], bit for bit: FP32 divisions, oracle's encoder."""
    x = x.cpu().float()
    x = x.t().contiguous() if transpose else x
    rows, cols = x.shape
    s = (block_amax(x, tile).numpy().astype(np.float32) / np.float32(448.0)).astype(np.float32)
    e = spread(torch.from_numpy(s), tile, rows, cols).numpy()
    with np.errstate(all="ignore"):
        v = np.where(e == 0, x.numpy(), x.numpy() / np.where(e == 0, np.float32(1), e)).astype(np.float32)
    q = np.zeros((rows, up(cols, 16)), np.uint8)
    q[:, :cols] = e4m3_encode(v)
    return q, s


def check_codes(codes, scales, want, err, what=""):
    """Block-scaled codes [rows, up(cols, 16)] of want [rows, cols], known to err:
    a scale is off by its block's largest err / 448 and one division's rounding,
    a quotient by one rounding more, a code by half a step."""
    rows, cols = want.shape
    s, s64 = scales.cpu().double().view(rows, -1), block_amax(want, False) / 448.0
    tol = block_amax(err, False) / 448.0 + s64 * 2 * U + 2.0 ** -149
    assert ((s - s64).abs() <= tol).all(), f"{what}: scales off by {((s - s64).abs() / tol).max():.3g} of the bound"
    got = decode(codes.view(rows, -1))
    assert (got[:, cols:] == 0).all(), f"{what}: padding"
    e = spread(s, False, rows, cols)
    live = e > 0
    t = torch.where(live, want / torch.where(live, e, torch.ones_like(e)), torch.zeros_like(want))
    d = torch.where(live, err / torch.where(live, e, torch.ones_like(e)), torch.zeros_like(want)) + t.abs() * 2 * U
    t = t.clamp(-448.0, 448.0)
    off = (got[:, :cols] - t).abs()
    tol = d + torch.maximum((t.abs() + d) * E4M3_HALF, torch.full_like(t, E4M3_SUB_HALF))
    assert (off <= tol).all(), f"{what}: {int((off > tol).sum())} codes outside, worst {(off / tol).max():.3g}"


def silu_mul(g, u):
    """(v, err).  The exponential takes a step (2 u), its correction and their
    product a rounding each, so d = 1 + p is within 5 u; the reciprocal and its
    Newton step 2 u, the two products u each: 9 u, held to 10.  Where the
    exponential overflows (g < -88.7) the result is a zero of at most 88.8 e^-88.7 |u|,
    below 2^-121 |u|."""
    g, u = g.cpu().double(), u.cpu().double()
    v = g * torch.sigmoid(g) * u
    return v, v.abs() * 10 * U + u.abs() * 2.0 ** -121


def linear(qx, qw, sx, sw, w_rows, bias=None, kind=0, residual=None):
    """(y, z, err, err_z).  A block's products are exact and their sum takes 8
    MFMA additions, the blocks' sums at most K / 128 FMAs and 16 additions of
    partial sums, each half a step of at most sum|terms|: (K/128 + 26) u is below
    1e-5 up to K = 18,000.  The scale of a block's sum is one FP32 number by
    definition.  act's slope is below 1.13."""
    a, b = decode(qx), decode(qw)
    (M, K), N = a.shape, b.shape[0]
    kb = up(K, BLOCK) // BLOCK
    sx, sw = sx.cpu().float().view(M, kb), sw.cpu().float()
    sw = sw.view(N, kb) if w_rows else sw.view(-1, kb).repeat_interleave(BLOCK, dim=0)[:N]
    z, terms = torch.zeros(M, N, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    for i in range(kb):
        c = slice(i * BLOCK, (i + 1) * BLOCK)
        alpha = (sx[:, i:i + 1] * sw[:, i].view(1, -1)).double()
        z += (a[:, c] @ b[:, c].t()) * alpha
        terms += (a[:, c].abs() @ b[:, c].abs().t()) * alpha.abs()
    assert kb <= 140
    err_z = 1e-5 * terms
    if bias is not None:
        z = z + bias.cpu().double()
    err_z = err_z + z.abs() * U
    y = act(z, kind)
    err = 1.13 * err_z + act_error(z, kind)
    if residual is not None:
        y = y + residual.cpu().double().view(M, N)
        err = err + y.abs() * U
    return y, z, err, err_z


def _gates(gate, rows):
    return 1.0 if gate is None else gate.cpu().double().view(-1, gate.shape[-1]).repeat_interleave(
        rows // (gate.numel() // gate.shape[-1]), dim=0)


def _row(p):
    return 1.0 if p is None else p.cpu().double()


def norm(x, w, h, gate, post, alpha, eps):
    """(y, r, rstd, post_rstd, err_y, err_r) of 2-D inputs, in 64 bits.

    A sum of H squares takes at most H/64 + 18 additions one after another and a
    rounding per square, relative to itself; the mean, the root and the division
    4 u.  v takes two products, the gate one, the FMA rounds r.  An error in r
    moves rstd by sum|r| err / sum r^2.  y takes two products."""
    x = x.cpu().double()
    rows, H = x.shape
    d = (H / 64 + 22) * U
    post_rstd, r, err_r = None, x, torch.zeros_like(x)
    if h is not None:
        v, e = h.cpu().double(), 0.0
        if post is not None:
            post_rstd = 1.0 / torch.sqrt(v.square().mean(dim=1) + eps)
            v, e = v * post_rstd[:, None] * _row(post), 0.5 * d + 6 * U
        v = alpha * _gates(gate, rows) * v
        r = x + v
        err_r = v.abs() * (e + 3 * U) + r.abs() * U
    rstd = 1.0 / torch.sqrt(r.square().mean(dim=1) + eps)
    y = r * rstd[:, None] * _row(w)
    moved = (r.abs() * err_r).sum(dim=1) / (r.square().sum(dim=1) + H * eps + 1e-300)
    err_rstd = 0.5 * d + 4 * U + moved
    err = y.abs() * (err_rstd[:, None] + 3 * U) + err_r * rstd[:, None] * (w.cpu().double().abs() if w is not None else 1.0)
    return y, r, rstd, post_rstd, err, err_r


def norm_backward(dy, r, w, rstd, h=None, gate=None, post=None, post_rstd=None, alpha=1.0, dr=None):
    """{name: (value, err)} for given FP32 rstd and post_rstd, in 64 bits.

    n, g and z round once each; a row's sums take H/64 + 20 additions, their
    products two roundings; dx's combination four, dr's addition one; p's factor
    three products and p one.  Sums over rows take at most rows + 20 additions."""
    dy, r, rs = dy.cpu().double(), r.cpu().double(), rstd.cpu().double().view(-1, 1)
    rows, H = r.shape
    d, many = (H / 64 + 24) * U, (rows + 24) * U
    n, g = r * rs, dy * _row(w)
    c, e1 = (g * n).mean(1, keepdim=True), d * (g * n).abs().mean(1, keepdim=True)
    dx = rs * (g - n * c)
    err = rs * (g.abs() * 4 * U + (n * c).abs() * 6 * U + n.abs() * e1) + dx.abs() * 2 * U
    if dr is not None:
        dx = dx + dr.cpu().double()
        err = err + dx.abs() * U
    out = {"dx": (dx, err)}
    if w is not None:
        out["dweight"] = ((dy * n).sum(0), many * (dy * n).abs().sum(0))
    if h is None:
        return out
    pr = 1.0 if post is None else post_rstd.cpu().double().view(-1, 1)
    z = h.cpu().double() * pr
    f = alpha * _gates(gate, rows) * _row(post)
    p = dx * f
    err_p = err * (f.abs() if torch.is_tensor(f) else abs(f)) + p.abs() * 4 * U
    if post is None:
        out["dhidden"] = (p, err_p)
    else:
        c2 = (p * z).mean(1, keepdim=True)
        e2 = d * (p * z).abs().mean(1, keepdim=True) + (err_p * z.abs()).mean(1, keepdim=True)
        dh = pr * (p - z * c2)
        out["dhidden"] = (dh, pr * (err_p + p.abs() * 2 * U + (z * c2).abs() * 6 * U + z.abs() * e2) + dh.abs() * 2 * U)
    a, ea = dx * z, err * z.abs() + (dx * z).abs() * 3 * U
    if gate is not None:
        by = lambda t: t.view(gate.numel() // H, -1, H).sum(1).view(gate.shape)  # noqa: E731
        k = alpha * _row(post)
        ka = k.abs() if torch.is_tensor(k) else abs(k)
        out["dgate"] = (by(a) * k, (by(ea) + (many + 3 * U) * by(a.abs())) * ka)
    if post is not None:
        k = alpha * _gates(gate, rows)
        ka = k.abs() if torch.is_tensor(k) else abs(k)
        out["dpost_weight"] = ((a * k).sum(0), ((ea + (many + 3 * U) * a.abs()) * ka).sum(0))
    return out
