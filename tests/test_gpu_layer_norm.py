"""GPU: the layer norm and its backward pass against 64-bit references
(bounds in norm_linear_ref)."""

import pytest
import torch

import mlp_fp8_quant_amd as fp8
import norm_linear_ref as ref

from gpu_util import device

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def make(rows, H, seed, xt=BF16, wt=BF16, shift=0.3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, H, generator=g) + shift
    x[torch.rand(rows, H, generator=g) < 0.005] *= 20
    w = 1 + 0.2 * torch.randn(H, generator=g)
    b = 0.3 * torch.randn(H, generator=g)
    d = device()
    return x.to(xt).to(d), w.to(wt).to(d), b.to(wt).to(d)


def check_forward(x, w, b, out_kind, eps=EPS, sy=None):
    y64, mean64, rstd64, err = ref.norm(x, w, b, eps)
    y, mean, rstd = fp8.fp8_layer_norm(x, w, b, eps, out_kind, sy, stats=True)
    if out_kind == fp8.OUT_FP8:
        ref.check_fp8(y, y64, err, sy, "y")
    else:
        ref.check(y, y64, err, "y")
    e_mean, e_rstd = ref.norm_errors(x.cpu().double(), eps)
    ref.check(mean, mean64, e_mean, "mean")
    ref.check(rstd, rstd64, rstd64 * e_rstd, "rstd")
    plain = fp8.fp8_layer_norm(x, w, b, eps, out_kind, sy)
    assert torch.equal(plain.view(torch.uint8), y.view(torch.uint8))


# widths around every vector, wave, workgroup and register limit
WIDTHS = [1, 2, 7, 8, 63, 64, 65, 128, 255, 512, 513, 1000, 1024, 1027, 2048, 2053, 4096, 4104, 5120, 8192, 8200,
          12288, 16384, 16392, 25600, 40001, 65536]


@pytest.mark.parametrize("H", WIDTHS)
def test_widths(H):
    sy = torch.tensor([0.02], device=device())
    for rows, xt, wt in ((3, BF16, F32), (5, F32, BF16)):
        x, w, b = make(rows, H, H, xt, wt)
        for out in (fp8.OUT_BF16, fp8.OUT_F32, fp8.OUT_FP8):
            check_forward(x, w, b, out, sy=sy)


@pytest.mark.parametrize("rows,H", [(1, 4096), (2, 5120), (255, 96), (1000, 1027), (2500, 264), (4099, 64), (5000, 24),
                                    (9000, 512), (3001, 2048)])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_rows(rows, H, xt):
    x, w, b = make(rows, H, rows, xt)
    check_forward(x, w, b, fp8.OUT_BF16)
    check_forward(x, w, b, fp8.OUT_FP8, sy=torch.tensor([0.01], device=device()))


def test_without_weight_or_bias():
    x, w, b = make(37, 1000, 1)
    for ww, bb in ((None, None), (w, None), (None, b)):
        check_forward(x, ww, bb, fp8.OUT_F32)
    x = x.view(37, 10, 100)
    assert fp8.fp8_layer_norm(x).shape == x.shape


@pytest.mark.parametrize("H", [96, 5120, 20000])
def test_large_means_and_constant_rows(H):
    # a mean far above the spread (squares' mean would cancel), a constant
    # row (variance 0 but for the mean's rounding) and a row of zeros
    d = device()
    x, w, b = make(6, H, 4, F32, F32)
    x = x * 0.1 + 1000.0
    x[2] = 0.75
    x[3] = 0.0
    check_forward(x, w, b, fp8.OUT_F32)
    for eps in (0.0, 1e-12, 0.1):
        check_forward(make(6, H, 5)[0], w, b, fp8.OUT_F32, eps)
    y = fp8.fp8_layer_norm(torch.zeros(2, H, device=d), w, b, 0.0, fp8.OUT_F32)
    assert bool(torch.isnan(y).all())      # 0 * (1 / sqrt 0)


def test_nan_and_infinite_rows_stay_alone():
    for rows, H in ((5, 4096), (3000, 512), (6, 777), (4, 30000)):
        x, w, b = make(rows, H, 6)
        y0 = fp8.fp8_layer_norm(x, w, b)
        x2 = x.clone()
        x2[1, H // 2] = float("nan")
        x2[3, H - 1] = float("inf")
        y, mean, rstd = fp8.fp8_layer_norm(x2, w, b, stats=True)
        bad = torch.zeros(rows, dtype=torch.bool, device=x.device)
        bad[[1, 3]] = True
        assert bool(torch.isnan(y[bad]).all()) and torch.equal(y[~bad], y0[~bad])
        assert torch.equal(torch.isnan(rstd), bad)
        q = fp8.fp8_layer_norm(x2, w, b, out_kind=fp8.OUT_FP8, sy=torch.tensor([0.01], device=x.device))
        assert bool((q[bad] == 0x7F).all()) and not bool((q[~bad] == 0x7F).any())


@pytest.mark.parametrize("rows,H", [(4, 4096), (300, 1027), (3000, 1024), (3, 40000)])
@pytest.mark.parametrize("xt,out", [(BF16, fp8.OUT_BF16), (F32, fp8.OUT_F32)])
def test_in_place(rows, H, xt, out):
    x, w, b = make(rows, H, 7, xt)
    want = fp8.fp8_layer_norm(x, w, b, out_kind=out)
    fp8.fp8_layer_norm(x, w, b, out_kind=out, out=x)
    assert torch.equal(x, want)


def test_empty():
    d = device()
    assert fp8.fp8_layer_norm(torch.empty(0, 64, device=d)).shape == (0, 64)
    assert fp8.fp8_layer_norm(torch.empty(5, 0, device=d)).shape == (5, 0)
    z = torch.empty(0, 64, device=d)
    s = torch.empty(0, device=d)
    dx, dw, db = fp8.fp8_layer_norm_backward(z, z, None, s, s)
    assert dx.shape == (0, 64) and not bool(dw.any()) and not bool(db.any()) and dw.shape == (64,)


@pytest.mark.parametrize("H", [61, 64, 1030, 4096, 8300])
def test_nothing_behind_the_outputs_is_written(H):
    d = device()
    x, w, b = make(9, H, 8)
    n = 9 * H
    for out, dtype in ((fp8.OUT_BF16, torch.int16), (fp8.OUT_F32, torch.int32), (fp8.OUT_FP8, torch.uint8)):
        buf = torch.full((n + 512,), 85, dtype=dtype, device=d)
        view = buf[:n] if out == fp8.OUT_FP8 else buf[:n].view({fp8.OUT_BF16: BF16, fp8.OUT_F32: F32}[out])
        fp8.fp8_layer_norm(x, w, b, out_kind=out, out=view, sy=torch.tensor([0.02], device=d))
        assert bool((buf[n:] == 85).all())
    dxb = torch.full((n + 512,), 85, dtype=torch.int16, device=d)
    dwb, dbb = (torch.full((H + 512,), 85, dtype=torch.int32, device=d) for _ in range(2))
    _, mean, rstd = fp8.fp8_layer_norm(x, w, b, stats=True)
    fp8.fp8_layer_norm_backward(x, x, w, mean, rstd, dx=dxb[:n].view(BF16), dweight=dwb[:H].view(F32),
                                dbias=dbb[:H].view(F32))
    assert all(bool((t[k:] == 85).all()) for t, k in ((dxb, n), (dwb, H), (dbb, H)))


def test_past_32_bit_offsets():
    d = device()
    rows, H = 530000, 4104                     # 2.2e9 elements
    x = torch.zeros(rows, H, dtype=BF16, device=d)
    tail, w, b = make(4, H, 9)
    x[-4:] = tail
    y64, _, _, err = ref.norm(tail, w, b, EPS)
    y, mean, rstd = fp8.fp8_layer_norm(x, w, b, stats=True)
    ref.check(y[-4:], y64, err)
    assert torch.equal(y[100], b)
    dy = torch.zeros(rows, H, dtype=BF16, device=d)
    dy[-4:] = tail.flip(0)
    dx, dw, db = fp8.fp8_layer_norm_backward(dy, x, w, mean, rstd, dx=dy)
    rx, rw, rb, ex, ew, eb = ref.norm_backward(tail.flip(0), tail, w, mean[-4:], rstd[-4:], None)
    ref.check(dx[-4:], rx, ex)
    ref.check(dw, rw, ew)
    ref.check(db, rb, eb)
    assert not bool(dx[:-4].any())


# ---------------------------------------------------------------------------
# Backward pass
# ---------------------------------------------------------------------------

def check_backward(rows, H, seed, xt=BF16, dt=BF16, wt=F32, dres=True, weight=True):
    x, w, b = make(rows, H, seed, xt, wt)
    w = w if weight else None
    g = torch.Generator().manual_seed(seed + 1)
    dy = torch.randn(rows, H, generator=g).to(dt).to(x.device)
    dr = torch.randn(rows, H, generator=g).to(xt).to(x.device) if dres else None
    _, mean, rstd = fp8.fp8_layer_norm(x, w, None, EPS, stats=True)
    got = fp8.fp8_layer_norm_backward(dy, x, w, mean, rstd, dres=dr)
    dx, dw, db, ex, ew, eb = ref.norm_backward(dy, x, w, mean, rstd, dr)
    ref.check(got[0], dx, ex, "dx")
    ref.check(got[1], dw, ew, "dweight")
    ref.check(got[2], db, eb, "dbias")
    again = fp8.fp8_layer_norm_backward(dy, x, w, mean, rstd, dres=dr)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    return dy, x, w, mean, rstd, dr, got


@pytest.mark.parametrize("H", WIDTHS)
def test_backward_widths(H):
    check_backward(3, H, H)
    check_backward(33, H, H + 1, F32, F32, BF16, dres=False)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 16, 17, 31, 32, 100, 513, 1500, 4096, 6000])
@pytest.mark.parametrize("H", [40, 512, 1027])
def test_backward_rows(rows, H):
    check_backward(rows, H, rows, dres=rows % 2 == 0)


@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("wt", [BF16, F32, None])
def test_backward_types(xt, dt, wt):
    check_backward(70, 520, 3, xt, dt, wt or F32, weight=wt is not None)
    check_backward(70, 521, 3, xt, dt, wt or F32, weight=wt is not None)


@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("H", [129, 135, 1536, 8185, 8192, 8193, 10001, 15361, 16384])
def test_backward_row_ends(xt, dt, H):
    # rows that end at each place of a group, a wave and a workgroup
    check_backward(5, H, H, xt, dt)


@pytest.mark.parametrize("H", [7, 100, 512, 700, 8192, 9000, 16384, 20000])
def test_backward_of_one_row(H):
    # one slab, whose sums are the results
    check_backward(1, H, H)


def test_backward_of_very_long_rows():
    # few slabs, since the columns fill the machine
    check_backward(40, 300007, 4)
    check_backward(1000, 17000, 5, F32, BF16, dres=False)


def test_widest_rows():
    # the widest row that the calls take, forward and backward
    d, H = device(), 1 << 26
    x = torch.randn(2, H, device=d).to(BF16)
    w = torch.randn(H, device=d).to(BF16)
    y, mean, rstd = fp8.fp8_layer_norm(x, w, None, EPS, out_kind=fp8.OUT_F32, stats=True)
    xd = x.double()
    m64 = xd.mean(1)
    r64 = ((xd - m64[:, None]).square().mean(1) + EPS).rsqrt()
    # a thread's sum of groups of eight keeps what its additions round off, so
    # a sum is within 3 (group) + 2 + 10 (lanes and waves) half steps of the sum of
    # its terms' sizes: 16 of 2^-24, and the squares' a few more
    assert bool(((mean - m64).abs() < 2.0 ** -20).all()) and bool(((rstd / r64 - 1).abs() < 2.0 ** -16).all())
    dx, dw, db = fp8.fp8_layer_norm_backward(x, x, w, mean, rstd)
    at = torch.tensor([0, 1, 8191, 8192, 1 << 20, H // 2, H - 9, H - 1], device=d)
    xh = (xd[:, at] - mean.double()[:, None]) * rstd.double()[:, None]
    assert torch.allclose(y[:, at].double(), xh * w[at].double(), rtol=2.0 ** -21, atol=2.0 ** -21)
    assert torch.allclose(dw[at].double(), (xd[:, at] * xh).sum(0), rtol=2.0 ** -20, atol=2.0 ** -20)
    assert torch.allclose(db[at].double(), xd[:, at].sum(0), rtol=2.0 ** -20, atol=2.0 ** -20)
    xa = (xd - mean.double()[:, None]) * rstd.double()[:, None]
    g = xd * w.double()
    want = (rstd.double()[:, None] * (g - g.mean(1, keepdim=True) - xa * (g * xa).mean(1, keepdim=True)))[:, at]
    # dx rounds to BF16; its two means are within 2^-19 of their terms' size
    assert torch.allclose(dx[:, at].double(), want, rtol=2.0 ** -8, atol=2.0 ** -8)


def test_backward_of_many_long_rows():
    check_backward(1100, 8200, 5)
    check_backward(600, 16384, 6, F32, F32, dres=False)


@pytest.mark.parametrize("H", [520, 1024, 1027, 9001, 16384, 30000])
def test_backward_in_place(H):
    dy, x, w, mean, rstd, dr, want = check_backward(65, H, 12)
    for over in ("dy", "dres", "x"):
        t = {"dy": dy.clone(), "x": x.clone(), "dres": dr.clone()}
        got = fp8.fp8_layer_norm_backward(t["dy"], t["x"], w, mean, rstd, dres=t["dres"], dx=t[over])
        assert all(torch.equal(p, q) for p, q in zip(got, want)), over


def test_backward_matches_differences():
    # <dx, v> against central differences of the 64-bit forward along v
    rows, H = 6, 300
    dy, x, w, mean, rstd, _, (dx, dw, db) = check_backward(rows, H, 13, F32, F32, F32, dres=False)
    g = torch.Generator().manual_seed(14)
    x64, w64 = x.cpu().double(), w.cpu().double()
    f = lambda a, c: (ref.norm(a, c, None, EPS)[0] * dy.cpu().double()).sum().item()  # noqa: E731
    h = 1e-5
    for _ in range(4):
        v = torch.randn(rows, H, generator=g, dtype=torch.float64)
        num = (f(x64 + h * v, w64) - f(x64 - h * v, w64)) / (2 * h)
        # FP32 entries: u-sized errors against sums of rows * H terms; the
        # differences' own error is O(h^2)
        assert abs((dx.cpu().double() * v).sum().item() - num) < 1e-4 * (dx.cpu().double() * v).abs().sum().item()
        c = torch.randn(H, generator=g, dtype=torch.float64)
        num = (f(x64, w64 + h * c) - f(x64, w64 - h * c)) / (2 * h)
        assert abs((dw.cpu().double() * c).sum().item() - num) < 1e-4 * (dw.cpu().double() * c).abs().sum().item()
