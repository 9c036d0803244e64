"""CPU: the refusals of the block-scaled FP8 calls and of the residual norm
before any device access, the binding's checks, the custom ops' fake kernels,
and the 64-bit references' gradients against differences.  No kernel runs."""

import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import block_norm_ref as ref
import mlp_fp8_quant_amd as fp8
import mlp_fp8_quant_amd.torch_ops  # noqa: F401
from mlp_fp8_quant_amd import _lib as L

P = ctypes.c_void_p
FAKE, ODD, NULL = P(0x10000), P(0x10004), P(0)     # never dereferenced: every call is refused first
OK, INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4, 6


def at(i, byte=0):
    return P((i << 20) + byte)             # a tensor of its own, 1 MiB apart


def call(f, full, args, plain=()):
    return f(**{k: v if k in plain else at(*v) if type(v) is tuple else at(v) for k, v in {**full, **args}.items()})


def quant(x=at(1), xe=0, q=at(2), s=at(3), M=4, K=20, tile=0, tr=0):
    return L.lib().fp8_quant_block(x, xe, q, s, M, K, tile, tr, NULL)


@pytest.mark.parametrize("want,args", [
    (INVALID, dict(xe=2)), (INVALID, dict(xe=-1)), (INVALID, dict(M=-1)), (INVALID, dict(K=-1)),
    (INVALID, dict(M=1 << 31)), (INVALID, dict(K=(1 << 26) + 1)), (INVALID, dict(tile=2)), (INVALID, dict(tr=-1)),
    (INVALID, dict(x=NULL)), (INVALID, dict(q=NULL)), (INVALID, dict(s=NULL)), (MISALIGNED, dict(x=at(1, 4))),
    (MISALIGNED, dict(q=at(2, 8))), (OK, dict(M=0, x=NULL, q=NULL, s=NULL)), (OK, dict(K=0, x=NULL)),
    # x is 4 x 20 BF16 = 160 bytes, q 4 x 32 = 128, transposed 20 x 16 = 320; scales 16, transposed 80, a tile 4
    (INVALID, dict(q=at(1, 144))), (INVALID, dict(q=at(3, -112))), (INVALID, dict(s=at(1, 156))),
    (INVALID, dict(s=at(2, 124))), (INVALID, dict(s=at(2, 316), tr=1)), (INVALID, dict(x=at(3, 64), tr=1)),
    (INVALID, dict(q=at(1, -112))), (INVALID, dict(x=at(2, 304), tr=1, tile=1)),
])
def test_quant_refusals(want, args):
    assert quant(**args) == want


def silu(g=at(1), u=at(4), q=at(2), s=at(3), M=4, K=20):
    return L.lib().silu_mul_2in_block(g, u, q, s, M, K, NULL)


@pytest.mark.parametrize("want,args", [
    (INVALID, dict(M=-1)), (INVALID, dict(K=(1 << 26) + 1)), (INVALID, dict(g=NULL)), (INVALID, dict(u=NULL)),
    (INVALID, dict(q=NULL)), (INVALID, dict(s=NULL)), (MISALIGNED, dict(g=at(1, 2))), (MISALIGNED, dict(u=at(4, 2))),
    (MISALIGNED, dict(q=at(2, 1))), (OK, dict(M=0, g=NULL)), (OK, dict(K=0, u=NULL)), (INVALID, dict(q=at(1))),
    (INVALID, dict(q=at(4, 144))), (INVALID, dict(s=at(4))), (INVALID, dict(s=at(2, 124)))])
def test_silu_refusals(want, args):
    assert silu(**args) == want


def linear(qx=FAKE, qw=FAKE, y=at(9), M=4, N=8, K=16, sx=FAKE, sw=FAKE, rows=0, bias=NULL, be=0, act=0,
           res=NULL, re=0, pre=NULL, out=0, sy=NULL):
    return L.lib().fp8_linear_block(qx, qw, y, M, N, K, sx, sw, rows, bias, be, act, res, re, pre, out, sy, NULL)


@pytest.mark.parametrize("want,args", [
    (UNSUPPORTED, dict(sx=NULL)), (UNSUPPORTED, dict(sw=NULL)), (UNSUPPORTED, dict(out=1)),
    (INVALID, dict(M=-1)), (INVALID, dict(N=-8)), (INVALID, dict(K=24)), (INVALID, dict(K=-16)),
    (INVALID, dict(out=3)), (INVALID, dict(out=-1)), (INVALID, dict(act=5)), (INVALID, dict(act=-1)),
    (INVALID, dict(rows=2)), (INVALID, dict(rows=-1)), (INVALID, dict(be=2)), (INVALID, dict(re=-1)),
    (INVALID, dict(qx=NULL)), (INVALID, dict(qw=NULL)), (INVALID, dict(y=NULL)), (INVALID, dict(M=1 << 31)),
    (INVALID, dict(K=8388576 + 16)), (INVALID, dict(N=0x7FFFF000 // 512)),
    (INVALID, dict(N=0x7FFFF000 // 1024, out=1, sy=FAKE, res=FAKE, re=1)),
    (MISALIGNED, dict(qx=ODD)), (MISALIGNED, dict(qw=ODD)), (MISALIGNED, dict(y=ODD)), (MISALIGNED, dict(bias=ODD)),
    (MISALIGNED, dict(res=ODD)), (MISALIGNED, dict(pre=ODD)),
    (OK, dict(M=0, qx=NULL, y=NULL)), (OK, dict(N=0, qw=NULL, y=NULL)), (INVALID, dict(M=0, act=9)),
])
def test_linear_refusals(want, args):
    assert linear(**args) == want


@pytest.mark.parametrize("args", [
    dict(y=1), dict(y=2), dict(y=4), dict(y=5), dict(y=6), dict(pre=1), dict(pre=2), dict(pre=3), dict(pre=4),
    dict(pre=7), dict(pre=5), dict(y=7, out=2), dict(y=7, out=1, sy=8), dict(y=8, out=1, sy=8), dict(pre=8, out=1, sy=8),
    dict(y=(7, 16)), dict(res=(3, 48)), dict(pre=(3, 16)), dict(sx=(3, 60)), dict(sw=(3, 60)), dict(bias=(3, 48)),
    dict(y=(5, 16), rows=1), dict(qx=(3, 48)), dict(qw=(3, 48))])
def test_linear_refuses_overlaps(args):
    # 1 qx, 2 qw, 3 y, 4 sx, 5 sw, 6 bias, 7 residual, 8 sy, 9 pre; y of 4 x 8 BF16 is 64 bytes
    assert call(linear, dict(qx=1, qw=2, y=3, sx=4, sw=5, bias=6, res=7, pre=9), args, ("out", "rows")) == INVALID


def norm(x=at(1), xe=0, h=at(2), he=0, gate=NULL, ge=0, gates=1, post=NULL, w=at(5), we=0, r=at(6), y=at(7), out=0,
         sy=NULL, s=NULL, rstd=NULL, prstd=NULL, rows=4, H=8, alpha=1.0, eps=1e-6):
    return L.lib().fp8_residual_norm(x, xe, h, he, gate, ge, gates, post, w, we, r, y, out, sy, s, rstd, prstd, rows,
                                     H, alpha, eps, NULL)


@pytest.mark.parametrize("want,args", [
    (INVALID, dict(xe=2)), (INVALID, dict(he=2)), (INVALID, dict(ge=2)), (INVALID, dict(we=2)), (INVALID, dict(out=4)),
    (INVALID, dict(out=-1)), (UNSUPPORTED, dict(out=1)), (INVALID, dict(out=3)), (INVALID, dict(rows=-1)),
    (INVALID, dict(H=-1)), (INVALID, dict(rows=1 << 31)), (INVALID, dict(H=(1 << 26) + 1)), (INVALID, dict(eps=-1e-6)),
    (INVALID, dict(eps=float("nan"))), (INVALID, dict(eps=float("inf"))), (INVALID, dict(alpha=float("nan"))),
    (INVALID, dict(alpha=float("inf"))), (INVALID, dict(x=NULL)), (INVALID, dict(y=NULL)), (INVALID, dict(r=NULL)),
    (INVALID, dict(h=NULL)), (INVALID, dict(h=NULL, r=NULL, gate=at(3))), (INVALID, dict(h=NULL, r=NULL, post=at(4))),
    (INVALID, dict(gate=at(3), gates=0)), (INVALID, dict(gate=at(3), gates=3)), (INVALID, dict(gate=at(3), gates=8)),
    (MISALIGNED, dict(x=at(1, 4))), (MISALIGNED, dict(h=at(2, 8))), (MISALIGNED, dict(gate=at(3, 4))),
    (MISALIGNED, dict(post=at(4, 4))), (MISALIGNED, dict(w=at(5, 4))), (MISALIGNED, dict(r=at(6, 4))),
    (MISALIGNED, dict(y=at(7, 4))), (OK, dict(rows=0, x=NULL, y=NULL)), (OK, dict(H=0)),
])
def test_norm_refusals(want, args):
    assert norm(**args) == want


@pytest.mark.parametrize("args", [
    dict(r=2), dict(r=3), dict(r=4), dict(r=5), dict(r=7), dict(r=(1, 16)), dict(y=1), dict(y=2), dict(y=3), dict(y=4),
    dict(y=5), dict(y=(6, 48)), dict(rstd=1), dict(rstd=2), dict(rstd=6), dict(rstd=7), dict(rstd=9), dict(prstd=1),
    dict(prstd=5), dict(prstd=7), dict(r=10, out=1, sy=10), dict(y=10, out=1, sy=10), dict(rstd=10, out=1, sy=10),
    dict(out=3, s=1), dict(out=3, s=2), dict(out=3, s=6), dict(out=3, s=(7, 60)), dict(out=3, s=8), dict(out=3, s=9)])
def test_norm_refuses_overlaps(args):
    # 1 x, 2 hidden, 3 gate, 4 post_weight, 5 weight, 6 r, 7 y, 8 rstd, 9 post_rstd
    full = dict(x=1, h=2, gate=3, post=4, w=5, r=6, y=7, rstd=8, prstd=9)
    assert call(norm, full, args, ("out",)) == INVALID


def back(dy=at(1), r=at(2), re=0, h=at(3), he=0, gate=at(4), ge=0, gates=2, post=at(5), w=at(6), we=0, rstd=at(7),
         prstd=at(8), dr=NULL, dx=at(10), dh=at(11), dg=at(12), dp=at(13), dw=at(14), rows=4, H=8, alpha=1.0, ws=at(15),
         wb=1 << 19):
    return L.lib().fp8_residual_norm_backward(dy, r, re, h, he, gate, ge, gates, post, w, we, rstd, prstd, dr, dx, dh,
                                              dg, dp, dw, rows, H, alpha, ws, wb, NULL)


@pytest.mark.parametrize("want,args", [
    (INVALID, dict(re=2)), (INVALID, dict(he=2)), (INVALID, dict(ge=2)), (INVALID, dict(we=2)), (INVALID, dict(rows=-2)),
    (INVALID, dict(H=-1)), (INVALID, dict(rows=1 << 31)), (INVALID, dict(alpha=float("nan"))), (INVALID, dict(gates=3)),
    (INVALID, dict(gates=0)), (INVALID, dict(dy=NULL)), (INVALID, dict(r=NULL)), (INVALID, dict(rstd=NULL)),
    (INVALID, dict(dx=NULL)), (INVALID, dict(dh=NULL)), (INVALID, dict(prstd=NULL)), (INVALID, dict(h=NULL)),
    (INVALID, dict(h=NULL, gate=NULL, dg=NULL, post=NULL, dp=NULL)), (INVALID, dict(gate=NULL)), (INVALID, dict(post=NULL)),
    *[(MISALIGNED, {k: at(20, 4)}) for k in ("dy", "r", "h", "gate", "post", "w", "dr", "dx", "dh", "dg", "dp", "dw")],
    (WORKSPACE, dict(ws=NULL)), (WORKSPACE, dict(ws=at(15, 4))), (WORKSPACE, dict(wb=16)),
    (OK, dict(H=0)), (OK, dict(rows=0, dg=NULL, dp=NULL, dw=NULL)),
])
def test_backward_refusals(want, args):
    assert back(**args) == want


@pytest.mark.parametrize("args", [
    dict(dx=3), dict(dx=4), dict(dx=5), dict(dx=6), dict(dx=7), dict(dx=8), dict(dx=11), dict(dx=12), dict(dx=(1, 16)),
    dict(dx=(2, 16)), dict(dx=(9, 48)), dict(dx=1, he=1), dict(dh=2), dict(dh=9), dict(dh=4), dict(dh=(3, 16)),
    dict(dh=(1, 16)), dict(dh=14), dict(dx=1, dh=1), dict(dg=1), dict(dg=4), dict(dg=9), dict(dg=13), dict(dp=5),
    dict(dp=3), dict(dp=14), dict(dw=6), dict(dw=7), dict(dw=2), dict(ws=1), dict(ws=8), dict(ws=10), dict(ws=14)])
def test_backward_refuses_overlaps(args):
    full = dict(dy=1, r=2, h=3, gate=4, post=5, w=6, rstd=7, prstd=8, dr=9, dx=10, dh=11, dg=12, dp=13, dw=14, ws=15)
    assert call(back, full, args, ("he",)) == INVALID


def test_backward_workspace():
    f = L.lib().fp8_residual_norm_backward_workspace
    assert f(1, 64, 1) == f(0, 64, 1) == f(64, 0, 1) == f(-1, 64, 1) == f(64, 64, 3) == f(64, 64, 0) == f(1 << 62, 64, 1) == 0
    assert f(4000, 64, 1) > 0 and f(4000, 64, 4000) >= 4000 * 2 * 64 * 4


def test_binding_refuses_before_the_library():
    q, s, b = torch.zeros(4, 16, dtype=torch.uint8), torch.ones(4), torch.zeros(4, 16, dtype=torch.bfloat16)
    for f in (lambda: fp8.fp8_quant_block(b), lambda: fp8.silu_mul_2in_block(b, b),
              lambda: fp8.fp8_linear_block(q, q, s, s), lambda: fp8.fp8_residual_norm(b, None, b),
              lambda: fp8.fp8_residual_norm_backward(b, b, None, s)):
        with pytest.raises(ValueError, match="must be on a GPU"):
            f()
    with pytest.raises(ValueError, match="go with hidden"):
        fp8.fp8_residual_norm(b, None, gate=s)
    with pytest.raises(ValueError, match="bfloat16 or torch.float32"):
        fp8.fp8_quant_block(q)
    with pytest.raises(TypeError):
        fp8.fp8_quant_block([1.0])


def test_binding_checks_shapes():
    with FakeTensorMode():
        e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        u8, bf = torch.uint8, torch.bfloat16
        qb = lambda **k: fp8.fp8_quant_block(**{**dict(x=e(4, 300)), **k})  # noqa: E731
        sb = lambda **k: fp8.silu_mul_2in_block(**{**dict(g=e(4, 40, t=bf), u=e(4, 40, t=bf)), **k})  # noqa: E731
        lin = lambda **k: fp8.fp8_linear_block(  # noqa: E731
            **{**dict(qx=e(4, 304, t=u8), qw=e(200, 304, t=u8), sx=e(4, 3), sw=e(2, 3)), **k})
        nm = lambda **k: fp8.fp8_residual_norm(**{**dict(x=e(4, 8), weight=e(8), hidden=e(4, 8)), **k})  # noqa: E731
        nb = lambda **k: fp8.fp8_residual_norm_backward(  # noqa: E731
            **{**dict(dy=e(4, 8), r=e(4, 8), weight=e(8), rstd=e(4), hidden=e(4, 8)), **k})
        for f, args, match in [
                (qb, dict(x=e(2, 2, 8), tile=True), "2-D"), (qb, dict(x=e(8, 4).t()), "contiguous"),
                (qb, dict(x=e()), "last"), (qb, dict(out=e(4, 300, t=u8)), "out must hold"),
                (qb, dict(scales=e(4, 2)), "scales must hold"), (qb, dict(out=e(300, 4, t=u8), transpose=True), "out must"),
                (sb, dict(u=e(4, 41, t=bf)), "same shape"), (sb, dict(g=e(4, 40)), "g must be"),
                (lin, dict(qw=e(200, 16, t=u8)), "shapes"), (lin, dict(sx=e(4)), "sx must hold"),
                (lin, dict(sw=e(200)), "sw must hold"), (lin, dict(sw=e(2, 3, t=bf)), "sw must be"),
                (lin, dict(bias=e(5)), "bias"), (lin, dict(residual=e(4, 5)), "residual"), (lin, dict(out_kind=3), "out_kind"),
                (lin, dict(pre=e(4, 200)), "pre must be"), (lin, dict(out=e(3, 200, t=bf)), "out must hold"),
                (nm, dict(weight=e(7)), "weight"), (nm, dict(hidden=e(4, 7)), "hidden"), (nm, dict(gate=e(7)), "gate"),
                (nm, dict(gate=e(3, 8)), "divide"), (nm, dict(gate=e(1, 4, 8)), "gate"),
                (nm, dict(post_weight=e(8, t=bf)), "post_weight must be"), (nm, dict(out_kind=4), "out_kind"),
                (nm, dict(stream_out=e(4, 8, t=bf)), "stream_out must be"), (nm, dict(x=e(8, 4).t()), "contiguous"),
                (nb, dict(dy=e(4, 7)), "dy must hold"), (nb, dict(hidden=e(4, 8, t=bf)), "hidden must be"),
                (nb, dict(rstd=e(3)), "one value per row"), (nb, dict(post_weight=e(8)), "post_rstd"),
                (nb, dict(dr=e(4, 8, t=bf)), "dr must be"), (nb, dict(dgate=e(8)), "dgate has no input"),
                (nb, dict(gate=e(2, 8), dgate=e(8)), "dgate must hold"), (nb, dict(dweight=e(7)), "dweight must"),
                (nb, dict(dy=None), "dy")]:
            with pytest.raises((ValueError, TypeError), match=match):
                f(**args)


def test_fake_kernels():
    ops = torch.ops.fp8mot
    with FakeTensorMode():
        e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        x = e(2, 5, 300, t=torch.bfloat16)
        q, s = ops.quant_block(x)
        assert q.shape == (2, 5, 304) and q.dtype == torch.uint8 and s.shape == (2, 5, 3)
        q, s = ops.quant_block(e(10, 300), True, True)
        assert q.shape == (300, 16) and s.shape == (3, 1)
        q, s = ops.silu_mul_block(x, x)
        assert q.shape == (2, 5, 304) and s.shape == (2, 5, 3)
        y = ops.linear_block(q, e(70, 304, t=torch.uint8), s, e(1, 3), None, 0, None, fp8.OUT_F32)
        assert y.shape == (2, 5, 70) and y.dtype == torch.float32
        y, r, rstd, post = ops.residual_norm(x, x, e(300), e(2, 300), e(300), 0.5, 1e-6, fp8.OUT_FP8, e(1))
        assert y.dtype == torch.uint8 and r.shape == x.shape and rstd.shape == post.shape == (2, 5)
        q, s, r = ops.residual_norm_block(x, x)
        assert q.shape == (2, 5, 304) and s.shape == (2, 5, 3) and r.dtype == x.dtype
        dx, dh, dw, dg, dp = ops.residual_norm_backward(x, r, e(300), rstd, x, e(2, 300), e(300), post)
        assert dx.shape == dh.shape == x.shape and dw.shape == dp.shape == (300,) and dg.shape == (2, 300)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gates", [0, 1, 3])
def test_reference_norm_gradient_against_differences(post, gates):
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    rows, H = 6, 11
    t = dict(x=r(rows, H), w=r(H), h=r(rows, H), gate=r(gates, H) if gates else None, post=r(H) if post else None)
    dy, dr = r(rows, H), r(rows, H)

    def loss(**k):
        v = {**t, **k}
        y, s, *_ = ref.norm(v["x"], v["w"], v["h"], v["gate"], v["post"], 0.3, 1e-6)
        return (y * dy).sum() + (s * dr).sum()

    _, s, rstd, prstd, _, _ = ref.norm(t["x"], t["w"], t["h"], t["gate"], t["post"], 0.3, 1e-6)
    out = ref.norm_backward(dy, s, t["w"], rstd, t["h"], t["gate"], t["post"], prstd, 0.3, dr)
    for name, of in (("dx", "x"), ("dhidden", "h"), ("dweight", "w"), ("dgate", "gate"), ("dpost_weight", "post")):
        if t[of] is None:
            assert name not in out
            continue
        flat, grad = t[of].reshape(-1), out[name][0].reshape(-1)
        for i in range(flat.numel()):
            d = torch.zeros_like(flat)
            d[i] = 1e-6
            num = (loss(**{of: t[of] + d.view(t[of].shape)}) - loss(**{of: t[of] - d.view(t[of].shape)})) / 2e-6
            assert abs(num - grad[i]) < 1e-6 * max(1.0, abs(grad[i])), (name, i)
