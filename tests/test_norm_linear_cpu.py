"""CPU: the C ABI's refusals of the Linear epilogue and the layer norm before
any device access, the binding's checks, the custom ops' fake kernels, and
the 64-bit references' gradients against differences.  No kernel runs."""

import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import mlp_fp8_quant_amd as fp8
import mlp_fp8_quant_amd.torch_ops  # noqa: F401
import norm_linear_ref as ref
from mlp_fp8_quant_amd import _lib as L

P = ctypes.c_void_p
FAKE, ODD, NULL = P(0x10000), P(0x10004), P(0)     # never dereferenced: every call is refused first
OK, INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4, 6


def linear(qx=FAKE, qw=FAKE, y=FAKE, M=4, N=8, K=16, sx=FAKE, sw=FAKE, rows=0, bias=NULL, be=0, act=0,
           res=NULL, re=0, pre=NULL, out=0, sy=NULL, accum=0, ws=NULL, wb=0):
    return L.lib().fp8_linear_act(qx, qw, y, M, N, K, sx, sw, rows, bias, be, act, res, re, pre, out, sy,
                                  accum, ws, wb, NULL)


@pytest.mark.parametrize("want,args", [
    (UNSUPPORTED, dict(sx=NULL)), (UNSUPPORTED, dict(sw=NULL)), (UNSUPPORTED, dict(out=1)),
    (INVALID, dict(M=-1)), (INVALID, dict(N=-8)), (INVALID, dict(K=24)), (INVALID, dict(K=-16)),
    (INVALID, dict(out=3)), (INVALID, dict(out=-1)), (INVALID, dict(accum=2)), (INVALID, dict(act=5)),
    (INVALID, dict(act=-1)), (INVALID, dict(rows=2)), (INVALID, dict(rows=-1)), (INVALID, dict(be=2)),
    (INVALID, dict(re=-1)), (INVALID, dict(qx=NULL)), (INVALID, dict(qw=NULL)), (INVALID, dict(y=NULL)),
    (INVALID, dict(M=1 << 31)), (INVALID, dict(K=8388576 + 16)), (INVALID, dict(N=0x7FFFF000 // 512)),
    (INVALID, dict(N=0x7FFFF000 // 1024, out=1, sy=FAKE, res=FAKE, re=1)),
    (MISALIGNED, dict(qx=ODD)), (MISALIGNED, dict(qw=ODD)), (MISALIGNED, dict(y=ODD)),
    (MISALIGNED, dict(bias=ODD)), (MISALIGNED, dict(res=ODD)), (MISALIGNED, dict(pre=ODD)),
    (MISALIGNED, dict(rows=1, sx=ODD)), (MISALIGNED, dict(rows=1, sw=ODD)),
    (OK, dict(M=0, qx=NULL, y=NULL)), (OK, dict(N=0, qw=NULL, y=NULL)),
    (INVALID, dict(M=0, act=9)),
])
def test_linear_refusals(want, args):
    assert linear(**args) == want


def test_linear_workspace_refusals():
    lib = L.lib()
    assert lib.fp8_linear_act_workspace(-1, 4, 16) == 0
    assert lib.fp8_linear_act_workspace(0, 4, 16) == 0
    for M, N, K in ((4, 8, 16), (16384, 25600, 5120), (1, 4096, 4096), (512, 4096, 12288)):
        assert lib.fp8_linear_act_workspace(M, N, K) == 0
    # K split over two, three and four workgroups
    for M, N, K, splits in ((7278, 290, 9984, 2), (3000, 700, 4000, 3), (578, 7537, 14240, 4)):
        need = lib.fp8_linear_act_workspace(M, N, K)
        assert need == splits * M * N * 4
        assert linear(M=M, N=N, K=K) == WORKSPACE
        assert linear(M=M, N=N, K=K, ws=FAKE, wb=need - 1) == WORKSPACE
        assert linear(M=M, N=N, K=K, ws=ODD, wb=need) == WORKSPACE


def linear_backward(dy=FAKE, pre=FAKE, act=1, dz=FAKE, db=FAKE, M=4, N=8, ws=FAKE, wb=1 << 30):
    return L.lib().fp8_linear_act_backward(dy, pre, act, dz, db, M, N, ws, wb, NULL)


@pytest.mark.parametrize("want,args", [
    (INVALID, dict(act=5)), (INVALID, dict(M=-1)), (INVALID, dict(N=-1)), (INVALID, dict(N=1 << 31)),
    (INVALID, dict(M=1 << 31)), (INVALID, dict(dy=NULL)), (INVALID, dict(pre=NULL)),
    (MISALIGNED, dict(dy=ODD)), (MISALIGNED, dict(pre=ODD)), (MISALIGNED, dict(dz=ODD)),
    (MISALIGNED, dict(db=ODD)), (WORKSPACE, dict(M=400, ws=NULL)), (WORKSPACE, dict(M=400, wb=16)),
    (WORKSPACE, dict(M=400, ws=ODD)), (OK, dict(N=0)), (OK, dict(M=0, db=NULL)), (OK, dict(dz=NULL, db=NULL)),
])
def test_linear_backward_refusals(want, args):
    assert linear_backward(**args) == want


def norm(x=FAKE, xe=0, w=FAKE, b=FAKE, wbe=0, y=FAKE, out=0, sy=NULL, mean=NULL, rstd=NULL, rows=4, H=8, eps=1e-5):
    return L.lib().fp8_layer_norm(x, xe, w, b, wbe, y, out, sy, mean, rstd, rows, H, eps, NULL)


@pytest.mark.parametrize("want,args", [
    (UNSUPPORTED, dict(out=1)), (INVALID, dict(out=3)), (INVALID, dict(xe=2)), (INVALID, dict(wbe=-1)),
    (INVALID, dict(rows=-1)), (INVALID, dict(H=-1)), (INVALID, dict(rows=1 << 31)), (INVALID, dict(H=1 << 31)),
    (INVALID, dict(eps=-1e-5)), (INVALID, dict(eps=float("nan"))), (INVALID, dict(eps=float("inf"))),
    (INVALID, dict(x=NULL)), (INVALID, dict(y=NULL)), (MISALIGNED, dict(x=ODD)), (MISALIGNED, dict(y=ODD)),
    (MISALIGNED, dict(w=ODD)), (MISALIGNED, dict(b=ODD)), (OK, dict(rows=0, x=NULL, y=NULL)), (OK, dict(H=0)),
])
def test_norm_refusals(want, args):
    assert norm(**args) == want


def norm_backward(dy=FAKE, de=0, x=FAKE, xe=0, w=FAKE, we=0, mean=FAKE, rstd=FAKE, dres=NULL, dx=FAKE, dw=FAKE,
                  db=FAKE, rows=4, H=8, ws=FAKE, wb=1 << 30):
    return L.lib().fp8_layer_norm_backward(dy, de, x, xe, w, we, mean, rstd, dres, dx, dw, db, rows, H, ws, wb, NULL)


@pytest.mark.parametrize("want,args", [
    (INVALID, dict(de=2)), (INVALID, dict(xe=2)), (INVALID, dict(we=2)), (INVALID, dict(rows=-1)),
    (INVALID, dict(H=-1)), (INVALID, dict(dy=NULL)), (INVALID, dict(x=NULL)), (INVALID, dict(mean=NULL)),
    (INVALID, dict(rstd=NULL)), (INVALID, dict(dx=NULL)), (MISALIGNED, dict(dy=ODD)), (MISALIGNED, dict(x=ODD)),
    (MISALIGNED, dict(w=ODD)), (MISALIGNED, dict(dres=ODD)), (MISALIGNED, dict(dx=ODD)),
    (MISALIGNED, dict(dw=ODD)), (MISALIGNED, dict(db=ODD)), (WORKSPACE, dict(rows=400, ws=NULL)),
    (WORKSPACE, dict(rows=400, wb=4)), (WORKSPACE, dict(rows=400, ws=ODD)), (WORKSPACE, dict(H=20000, ws=NULL)),
    (OK, dict(H=0)), (OK, dict(rows=0, dw=NULL, db=NULL)),
])
def test_norm_backward_refusals(want, args):
    assert norm_backward(**args) == want


def at(i, byte=0):
    return P((i << 20) + byte)             # a tensor of its own, 1 MiB apart


@pytest.mark.parametrize("args", [
    dict(y=1), dict(y=2), dict(y=4), dict(y=5), dict(y=6), dict(pre=1), dict(pre=2), dict(pre=3), dict(pre=4),
    dict(pre=7), dict(pre=5), dict(y=7, out=2), dict(y=7, out=1, sy=8), dict(y=8, out=1, sy=8), dict(pre=8, out=1, sy=8),
    dict(y=(7, 16)), dict(res=(3, 48)), dict(pre=(3, 16)), dict(rows=1, y=(4, 0)), dict(bias=(3, 48)),
    dict(qx=(3, 48)), dict(qw=(3, 48))])
def test_linear_refuses_overlaps(args):
    # 1 qx, 2 qw, 3 y, 4 sx, 5 sw, 6 bias, 7 residual, 8 sy, 9 pre; y of 4 x 8 BF16 is 64 bytes
    full = dict(qx=1, qw=2, y=3, sx=4, sw=5, bias=6, res=7, pre=9)
    a = {k: v if k in ("out", "rows") else at(*v) if type(v) is tuple else at(v) for k, v in {**full, **args}.items()}
    assert linear(**a) == INVALID


@pytest.mark.parametrize("args", [
    dict(dz=(1, 16)), dict(dz=(2, 48)), dict(db=1), dict(db=2), dict(db=3), dict(db=(3, 48)), dict(dy=(3, 32))])
def test_linear_backward_refuses_overlaps(args):
    full = dict(dy=1, pre=2, dz=3, db=4)
    assert linear_backward(**{k: at(*v) if type(v) is tuple else at(v) for k, v in {**full, **args}.items()}) == INVALID


@pytest.mark.parametrize("args", [
    dict(y=2), dict(y=3), dict(y=4), dict(y=5), dict(y=(1, 16)), dict(y=1, out=2), dict(y=1, xe=1), dict(mean=1),
    dict(mean=5), dict(mean=2), dict(rstd=6), dict(rstd=3), dict(y=7, out=1, sy=7), dict(mean=7, out=1, sy=7)])
def test_norm_refuses_overlaps(args):
    full = dict(x=1, w=2, b=3, mean=4, rstd=5, y=6)
    a = {k: v if k in ("out", "xe") else at(*v) if type(v) is tuple else at(v) for k, v in {**full, **args}.items()}
    assert norm(**a) == INVALID


@pytest.mark.parametrize("args", [
    dict(dx=3), dict(dx=4), dict(dx=5), dict(dx=8), dict(dx=(1, 16)), dict(dx=(2, 16)), dict(dx=(6, 16)), dict(dx=1, de=1),
    dict(dw=1), dict(dw=2), dict(dw=3), dict(dw=4), dict(dw=6), dict(dw=9), dict(db=7), dict(db=5), dict(db=2)])
def test_norm_backward_refuses_overlaps(args):
    # 1 dy, 2 x, 3 weight, 4 mean, 5 rstd, 6 dres, 7 dx, 8 dweight, 9 dbias
    full = dict(dy=1, x=2, w=3, mean=4, rstd=5, dres=6, dx=7, dw=8, db=9)
    a = {k: v if k == "de" else at(*v) if type(v) is tuple else at(v) for k, v in {**full, **args}.items()}
    assert norm_backward(**a) == INVALID


def test_backward_workspaces():
    lib, huge = L.lib(), 1 << 62
    for f in (lib.fp8_linear_act_backward_workspace, lib.fp8_layer_norm_backward_workspace):
        # one slab of rows writes its sums where they belong; refused sizes need nothing
        assert f(4, 64) == f(0, 64) == f(64, 0) == f(-1, 64) == f(huge, 64) == f(64, huge) == 0
        assert f(4000, 64) > 0
    assert lib.fp8_linear_act_workspace(huge, 64, 64) == lib.fp8_linear_act_workspace(64, huge, 64) == 0


def test_binding_refuses_before_the_library():
    # CPU tensors and wrong types never reach the library
    q = torch.zeros(4, 16, dtype=torch.uint8)
    s = torch.ones(1)
    for call in (lambda: fp8.fp8_linear_act(q, q, s, s), lambda: fp8.fp8_layer_norm(torch.zeros(4, 16)),
                 lambda: fp8.fp8_linear_act_backward(torch.zeros(4, 16, dtype=torch.bfloat16), None),
                 lambda: fp8.fp8_layer_norm_backward(torch.zeros(4, 16), torch.zeros(4, 16), None, s, s)):
        with pytest.raises(ValueError, match="must be on a GPU"):
            call()
    for bad in (torch.zeros(4, 16, dtype=torch.float16), torch.zeros(4, 16, dtype=torch.int32)):
        with pytest.raises(ValueError, match="bfloat16 or torch.float32"):
            fp8.fp8_layer_norm(bad)
    with pytest.raises(TypeError):
        fp8.fp8_layer_norm([1.0, 2.0])


def test_binding_checks_shapes():
    # shape checks come before any device access: fake CUDA tensors will do
    with FakeTensorMode():
        e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        u8, bf = torch.uint8, torch.bfloat16
        qx, qw, s = e(4, 32, t=u8), e(6, 32, t=u8), e(1)
        lin = lambda **k: fp8.fp8_linear_act(**{**dict(qx=qx, qw=qw, sx=s, sw=s), **k})  # noqa: E731
        ln = lambda **k: fp8.fp8_layer_norm(**{**dict(x=e(4, 8), weight=e(8)), **k})  # noqa: E731
        lb = lambda **k: fp8.fp8_layer_norm_backward(  # noqa: E731
            **{**dict(dy=e(4, 8), x=e(4, 8), weight=e(8), mean=e(4), rstd=e(4)), **k})
        ab = lambda **k: fp8.fp8_linear_act_backward(**{**dict(dy=e(4, 8, t=bf), pre=e(4, 8, t=bf)), **k})  # noqa: E731
        for call, args, match in [
                (lin, dict(qw=e(6, 16, t=u8)), "shapes"), (lin, dict(bias=e(5)), "bias"),
                (lin, dict(bias=e(6, t=torch.float16)), "bias"), (lin, dict(residual=e(4, 5)), "residual"),
                (lin, dict(residual=e(6, 4).t()), "contiguous"), (lin, dict(rowwise=True), "one scale per row"),
                (lin, dict(sx=e(4)), "exactly one"), (lin, dict(out=e(4, 6)), "out must be"),
                (lin, dict(out_kind=7), "out_kind"), (lin, dict(pre=e(4, 6)), "pre must be"),
                (lin, dict(pre=e(3, 6, t=bf)), "pre must hold"), (lin, dict(out=e(3, 6, t=bf)), "out must hold"),
                (ln, dict(weight=e(7)), "weight"), (ln, dict(bias=e(9)), "bias"),
                (ln, dict(bias=e(8, t=bf)), "bias must be"), (ln, dict(x=e(8, 4).t()), "contiguous"),
                (ln, dict(out=e(4, 8)), "out must be"), (ln, dict(x=e()), "last"),
                (lb, dict(dy=e(4, 7)), "dy must hold"), (lb, dict(dres=e(4, 8, t=bf)), "dres must be"),
                (lb, dict(mean=e(3)), "one value per row"), (lb, dict(dweight=e(7)), "dweight"),
                (lb, dict(dx=e(4, 8, t=bf)), "dx must be"), (lb, dict(dy=None), "dy"),
                (ab, dict(pre=e(4, 7, t=bf)), "pre must hold"), (ab, dict(dy=e(4, 8)), "dy must be"),
                (ab, dict(dbias=e(7)), "dbias"), (ab, dict(dz=e(3, 8, t=bf)), "dz must hold")]:
            with pytest.raises(ValueError, match=match):
                call(**args)


def test_fake_kernels():
    ops = torch.ops.fp8mot
    with FakeTensorMode():
        e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        x = e(2, 5, 64, t=torch.bfloat16)
        q, mean, rstd = ops.layer_norm(x, e(64), e(64), 1e-5, fp8.OUT_FP8, e(1))
        assert q.shape == x.shape and q.dtype == torch.uint8 and mean.shape == rstd.shape == (2, 5)
        w = e(96, 64, t=torch.uint8)
        y = ops.linear_act(q, w, e(1), e(1), e(96), fp8.ACT_SILU, None, fp8.OUT_F32)
        assert y.shape == (2, 5, 96) and y.dtype == torch.float32
        y, pre = ops.linear_act_train(q, w, e(1), e(1), e(96), fp8.ACT_SILU)
        assert y.dtype == pre.dtype == torch.bfloat16 and pre.shape == (2, 5, 96)
        dz, db = ops.linear_act_backward(y, pre, fp8.ACT_SILU)
        assert dz.shape == y.shape and db.shape == (96,) and db.dtype == torch.float32
        dx, dw, db = ops.layer_norm_backward(x, x, e(64), mean, rstd, x)
        assert dx.shape == x.shape and dx.dtype == x.dtype and dw.shape == db.shape == (64,)


@pytest.mark.parametrize("kind", ref.ACTS)
def test_reference_slopes_against_differences(kind):
    z = torch.linspace(-6, 6, 241, dtype=torch.float64) + 0.0123
    h = 1e-6
    num = (ref.act(z + h, kind) - ref.act(z - h, kind)) / (2 * h)
    # h^2 times a third derivative below 3, and 1e-16 |act| / h
    assert torch.allclose(ref.act_slope(z, kind), num, rtol=0, atol=2e-9)


def test_reference_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, dy = r(3, 17), r(17), r(3, 17)
    _, mean, rstd, _ = ref.norm(x, w, None, 1e-5)
    dx, dw, db, *_ = ref.norm_backward(dy, x, w, mean, rstd, None)
    f = lambda a, c, e: (ref.norm(a, c, e, 1e-5)[0] * dy).sum()  # noqa: E731
    h, b = 1e-6, r(17)
    for i in range(17):
        d = torch.zeros(17, dtype=torch.float64)
        d[i] = h
        assert abs((f(x, w + d, b) - f(x, w - d, b)) / (2 * h) - dw[i]) < 1e-8
        assert abs((f(x, w, b + d) - f(x, w, b - d)) / (2 * h) - db[i]) < 1e-8
        for row in range(3):
            e = torch.zeros(3, 17, dtype=torch.float64)
            e[row, i] = h
            assert abs((f(x + e, w, b) - f(x - e, w, b)) / (2 * h) - dx[row, i]) < 1e-7
