"""GPU: the norms before and after a block with its gate and residual scale,
forward and backward, against the 64-bit formulas."""

import pytest
import torch

import block_norm_ref as ref
import mlp_fp8_quant_amd as fp8

from gpu_util import device
from norm_linear_ref import check_fp8

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
# one column to rows beyond registers; rows that end inside a group of eight, sixteen and a block
WIDTHS = [1, 8, 100, 128, 129, 512, 520, 1027, 4096, 5120, 8192, 8200, 16384, 16393]


def inputs(rows, H, xt, ht, wt, gates, post, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=(2 * r(rows, H)).to(xt), h=r(rows, H).to(ht), w=(1 + 0.2 * r(H)).to(wt),
                gate=r(gates, H).to(wt) if gates else None, post=(1 + 0.2 * r(H)).to(wt) if post else None,
                dy=r(rows, H).to(ht), dr=r(rows, H).to(xt))


def dev(t):
    return None if t is None else t.to(device())


def run(t, **k):
    return fp8.fp8_residual_norm(dev(t["x"]), dev(t["w"]), dev(t["h"]), gate=dev(t["gate"]), post_weight=dev(t["post"]),
                                 **k)


def check_forward(t, alpha, eps=1e-6):
    y64, r64, rs, prs, err, err_r = ref.norm(t["x"], t["w"], t["h"], t["gate"], t["post"], alpha, eps)
    H = t["x"].shape[-1]
    y, r, rstd, prstd = run(t, alpha=alpha, eps=eps, out_kind=fp8.OUT_F32, stats=True)
    ref.check(y, y64, err, "y")
    ref.check(r, r64, err_r, "r")
    rel = err.amax() * 0 + (H / 64 + 40) * ref.U
    moved = (r64.abs() * err_r).sum(1) / (r64.square().sum(1) + H * eps)
    ref.check(rstd, rs, rs * (rel + moved), "rstd")
    assert (prstd is None) == (prs is None)
    if prs is not None:
        ref.check(prstd, prs, prs * rel, "post_rstd")
    ref.check(run(t, alpha=alpha, eps=eps)[0], y64, err, "bf16")
    sy = torch.tensor([0.02])
    q, r2 = run(t, alpha=alpha, eps=eps, out_kind=fp8.OUT_FP8, sy=sy.to(device()))
    check_fp8(q, y64, err, sy, "fp8")
    assert torch.equal(r, r2)
    (q, s), _ = run(t, alpha=alpha, eps=eps, out_kind=fp8.OUT_FP8_BLOCK)
    ref.check_codes(q, s, y64, err, "block")


def check_backward(t, alpha, dr=True):
    _, r, rstd, prstd = run(t, alpha=alpha, stats=True)
    d = t["dr"] if dr else None
    want = ref.norm_backward(t["dy"], r, t["w"], rstd, t["h"], t["gate"], t["post"], prstd, alpha, d)
    got = fp8.fp8_residual_norm_backward(dev(t["dy"]), r, dev(t["w"]), rstd, dev(t["h"]), gate=dev(t["gate"]),
                                         post_weight=dev(t["post"]), post_rstd=prstd, alpha=alpha, dr=dev(d))
    for name, v in zip(("dx", "dhidden", "dweight", "dgate", "dpost_weight"), got):
        assert (v is None) == (name not in want), name
        if v is not None:
            ref.check(v, *want[name], name)


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("rows", [1, 6])
def test_widths(rows, H):
    t = inputs(rows, H, BF16, BF16, BF16, 1, True, H)
    check_forward(t, 0.5)
    check_backward(t, 0.5)


@pytest.mark.parametrize("H", [40, 300, 1027, 8200])
@pytest.mark.parametrize("xt,ht,wt", [(BF16, F32, F32), (F32, BF16, BF16), (F32, F32, F32), (BF16, BF16, F32)])
@pytest.mark.parametrize("gates,post", [(0, False), (1, False), (0, True), (4, True), (12, False), (12, True)])
def test_types_gates_and_norms(gates, post, xt, ht, wt, H):
    t = inputs(12, H, xt, ht, wt, gates, post, gates + H)
    check_forward(t, 0.22)
    check_backward(t, 0.22, dr=post)


@pytest.mark.parametrize("rows,H", [(64, 4096), (130, 1027), (513, 100), (700, 520), (2000, 33), (300, 5120), (90, 8200)])
@pytest.mark.parametrize("gates", [0, 1, 2])
def test_many_rows(rows, H, gates):
    rows += rows % 2
    t = inputs(rows, H, BF16, BF16, F32, gates, gates != 1, rows)
    check_forward(t, 1.0)
    check_backward(t, 1.0)


@pytest.mark.parametrize("H", [64, 1000, 9000])
@pytest.mark.parametrize("gates", [250, 500])
def test_a_gate_for_each_few_rows(gates, H):
    t = inputs(500, H, BF16, BF16, BF16, gates, True, H)
    check_forward(t, 1.0)
    check_backward(t, 1.0)


@pytest.mark.parametrize("gates,per,H", [(16390, 1, 33), (16384, 3, 128), (4100, 2, 500), (1540, 3, 600), (1700, 1, 1027),
                                         (520, 2, 4096), (515, 1, 5123), (700, 1, 7000), (513, 2, 8200), (41, 1, 200001)])
@pytest.mark.parametrize("xt,wt,post", [(BF16, BF16, True), (F32, F32, False)])
def test_many_gates(gates, per, H, xt, wt, post):
    # gates share a workgroup's sums
    t = inputs(gates * per, H, xt, BF16, wt, gates, post, H)
    check_forward(t, 0.5)
    check_backward(t, 0.5, dr=post)


@pytest.mark.parametrize("H", [7, 128, 1030, 9000])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_without_hidden(xt, H):
    t = inputs(5, H, xt, xt, F32, 0, False, H)
    y64, _, rs, _, err, _ = ref.norm(t["x"], t["w"], None, None, None, 1.0, 1e-6)
    y, r, rstd, prstd = fp8.fp8_residual_norm(dev(t["x"]), dev(t["w"]), stats=True, out_kind=fp8.OUT_F32)
    assert r is None and prstd is None
    ref.check(y, y64, err)
    (q, s), _ = fp8.fp8_residual_norm(dev(t["x"]), dev(t["w"]), out_kind=fp8.OUT_FP8_BLOCK)
    ref.check_codes(q, s, y64, err)
    want = ref.norm_backward(t["dy"], t["x"], t["w"], rstd, dr=t["dr"])
    got = fp8.fp8_residual_norm_backward(dev(t["dy"]), dev(t["x"]), dev(t["w"]), rstd, dr=dev(t["dr"]))
    assert got[1] is None and got[3] is None and got[4] is None
    ref.check(got[0], *want["dx"])
    ref.check(got[2], *want["dweight"])
    y, _ = fp8.fp8_residual_norm(dev(t["x"]), None, out_kind=fp8.OUT_F32)          # no weight: ones
    y64, *_, err, _ = ref.norm(t["x"], None, None, None, None, 1.0, 1e-6)
    ref.check(y, y64, err)
    assert fp8.fp8_residual_norm_backward(dev(t["dy"]), dev(t["x"]), None, rstd)[2] is None


@pytest.mark.parametrize("H", [24, 600, 5120, 9000])
def test_in_place(H):
    t = inputs(9, H, BF16, BF16, BF16, 3, True, H)
    y, r, rstd, prstd = run(t, stats=True)
    x = dev(t["x"])
    y2, r2 = fp8.fp8_residual_norm(x, dev(t["w"]), dev(t["h"]), gate=dev(t["gate"]), post_weight=dev(t["post"]),
                                   stream_out=x)
    assert r2.data_ptr() == x.data_ptr() and torch.equal(r, x) and torch.equal(y, y2)
    args = dict(gate=dev(t["gate"]), post_weight=dev(t["post"]), post_rstd=prstd)
    want = fp8.fp8_residual_norm_backward(dev(t["dy"]), r, dev(t["w"]), rstd, dev(t["h"]), dr=dev(t["dr"]), **args)
    dy, h, dr = dev(t["dy"]), dev(t["h"]), dev(t["dr"])
    for dx, dh in ((dr, h), (dy, h), (r.clone(), dy)):
        dy_, h_, dr_ = dy.clone(), h.clone(), dr.clone()
        names = {dy.data_ptr(): dy_, h.data_ptr(): h_, dr.data_ptr(): dr_}
        r_ = dx if dx.data_ptr() not in names else r
        got = fp8.fp8_residual_norm_backward(dy_, r_, dev(t["w"]), rstd, h_, dr=dr_, dx=names.get(dx.data_ptr(), dx),
                                             dhidden=names[dh.data_ptr()], **args)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("H", [128, 1000, 9000])
def test_rows_of_zeros_and_of_nothing_else(H):
    # padding: zero rows give zeros, a zero scale, and no gradient of their own; eps 0 makes them NaN
    t = inputs(4, H, BF16, BF16, BF16, 1, True, 1)
    t["x"][1], t["h"][1] = 0.0, 0.0
    (q, s), r, rstd, _ = run(t, out_kind=fp8.OUT_FP8_BLOCK, stats=True)
    assert (q[1] == 0).all() and (s[1] == 0).all() and (r[1] == 0).all()
    check_forward(t, 1.0)
    check_backward(t, 1.0)
    y, _ = run(t, eps=0.0)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[0]).all()


@pytest.mark.parametrize("H", [128, 1000, 9000])
@pytest.mark.parametrize("odd", [float("nan"), float("inf")])
def test_nan_and_infinities_stay_in_their_rows(odd, H):
    t = inputs(5, H, BF16, BF16, BF16, 1, True, 2)
    (cq, cs), cr = run(t, out_kind=fp8.OUT_FP8_BLOCK)
    t["h"][2, H // 2] = odd
    t["x"][4, 0] = odd
    (q, s), r = run(t, out_kind=fp8.OUT_FP8_BLOCK)
    for i in (0, 1, 3):
        assert torch.equal(q[i], cq[i]) and torch.equal(s[i], cs[i]) and torch.equal(r[i], cr[i])
    assert torch.isnan(s[2]).any() and torch.isnan(s[4]).any()


@pytest.mark.parametrize("H", [128, 1027, 9000])
def test_empty_batches(H):
    t = inputs(0, H, BF16, BF16, BF16, 2, True, 0)
    y, r = run(t)
    assert y.shape == r.shape == (0, H)
    z = torch.zeros(0, device=device())
    got = fp8.fp8_residual_norm_backward(dev(t["dy"]), dev(t["x"]), dev(t["w"]), z, dev(t["h"]), gate=dev(t["gate"]),
                                         post_weight=dev(t["post"]), post_rstd=z)
    assert got[0].shape == (0, H) and all((g == 0).all() for g in got[2:]) and got[3].shape == (2, H)


def test_ranks_and_a_flat_gate():
    t = inputs(24, 264, BF16, BF16, F32, 1, True, 4)
    (q, s), r = run(t, out_kind=fp8.OUT_FP8_BLOCK)
    t3 = {**t, "x": t["x"].view(2, 12, 264), "h": t["h"].view(2, 12, 264), "gate": t["gate"].view(264)}
    (q3, s3), r3, rstd, prstd = run(t3, out_kind=fp8.OUT_FP8_BLOCK, stats=True)
    assert q3.shape == (2, 12, 272) and s3.shape == (2, 12, 3) and rstd.shape == prstd.shape == (2, 12)
    assert torch.equal(q3.view(24, 272), q) and torch.equal(s3.view(24, 3), s) and torch.equal(r3.view(24, 264), r)
    got = fp8.fp8_residual_norm_backward(dev(t3["x"]), r3, dev(t["w"]), rstd, dev(t3["h"]), gate=dev(t3["gate"]),
                                         post_weight=dev(t["post"]), post_rstd=prstd)
    assert got[0].shape == (2, 12, 264) and got[3].shape == (264,)


def test_widest_rows():
    # as many columns as the calls take.  In each result a value is off by a handful of FP32 roundings (at most 12, 16
    # counted) of the magnitudes that are added for it; dx and r by their BF16 rounding besides.
    H, rows, U, alpha = 2 ** 26, 2, 2.0 ** -24, 0.5
    g = torch.Generator(device=device()).manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device=device())  # noqa: E731
    x, h, dy = (r(rows, H).to(BF16) for _ in range(3))
    w, gate, post = (1 + 0.1 * r(H) for _ in range(3))

    def close(got, want, size, half=0.0):
        for a, b, c in zip(got.view(-1, H), want.view(-1, H), size.view(-1, H)):
            assert ((a.double() - b).abs() <= 16 * U * c + half * b.abs()).all()

    y, got_r, rstd, prstd = fp8.fp8_residual_norm(x, w, h, gate=gate, post_weight=post, alpha=alpha, out_kind=fp8.OUT_F32,
                                                  stats=True)
    f = alpha * gate.double() * post.double()
    rms = lambda t: (t * t).mean(-1, keepdim=True).add(1e-6).rsqrt()  # noqa: E731
    prs = rms(h.double())
    v = h.double() * prs * f
    r64 = x.double() + v
    rs = rms(r64)
    size = x.double().abs() + v.abs()
    assert ((prstd.double() * prs.reciprocal().view(-1) - 1).abs() <= 16 * U).all()
    assert ((rstd.double() * rs.reciprocal().view(-1) - 1).abs() <= 16 * U).all()
    close(y, r64 * rs * w, size * rs * w.abs())
    close(got_r, r64, size, 2.0 ** -8)
    del y, v, r64, size
    dx, dh, dw, dgate, dpost = fp8.fp8_residual_norm_backward(dy, got_r, w, rstd, h, gate=gate, post_weight=post,
                                                              post_rstd=prstd, alpha=alpha)
    n = got_r.double() * rstd.double().view(-1, 1)
    gw = dy.double() * w.double()
    c = (gw * n).mean(-1, keepdim=True)
    rs = rstd.double().view(-1, 1)
    # (c is off by some 2^-24 of the mean magnitude, about 1)
    dx64, size = rs * (gw - n * c), rs * (gw.abs() + n.abs())
    close(dx, dx64, size, 2.0 ** -8)
    close(dw, (dy.double() * n).sum(0), (dy.double() * n).abs().sum(0))
    del gw, n
    z = h.double() * prstd.double().view(-1, 1)
    zx, zs = (dx64 * z).sum(0), (size * z.abs()).sum(0)
    close(dgate, alpha * post.double() * zx, alpha * post.double().abs() * zs)
    close(dpost, alpha * gate.double() * zx, alpha * gate.double().abs() * zs)
    p = dx64 * f
    c2 = (p * z).mean(-1, keepdim=True)
    prs = prstd.double().view(-1, 1)
    close(dh, prs * (p - z * c2), prs * (size * f.abs() + z.abs()), 2.0 ** -8)
