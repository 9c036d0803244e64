"""GPU: the layer norm and its backward pass where range and rounding bite:
rows whose mean is far above their spread, wide FP32 rows, backward passes
whose statistics leave FP32's range in columns past the row's end.  References
are 64-bit, from the formulas."""

import pytest
import torch

import mlp_fp8_quant_amd as fp8
import norm_linear_ref as ref

from gpu_util import device

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = ref.U


# ---------------------------------------------------------------------------
# Means far above the spread
# ---------------------------------------------------------------------------

# (rows, H): each kernel of the forward pass, whole and ragged rows: 16 and 64
# threads, one to four groups of eight per thread, three reads of the row
SHAPES = [(5, 7), (700, 96), (700, 128), (5, 300), (700, 512), (9, 1027), (700, 1000), (700, 2048), (600, 4096),
          (600, 4104), (700, 5120), (600, 6144), (600, 8192), (600, 9001), (550, 12288), (7, 5120), (7, 16384),
          (600, 16000), (6, 20000), (6, 32768), (5, 40001)]
# additions one after another in any of a row's sums: 32 of a thread's, four
# inside 16 lanes, two over the wave, 15 over the waves, and the products
DEPTH = 60 * U


def corrected_errors(x):
    """Bounds for a row whose mean is taken twice: first a sum of x, off by
    e0, then the mean of the differences from it, which corrects mean and
    variance.  Only the differences' roundings remain: of mean x as xh uses it
    (absolute), and of the variance (absolute)."""
    mean = x.mean(dim=-1, keepdim=True)
    spread = (x - mean).abs().mean(dim=-1)
    e0 = DEPTH * x.abs().mean(dim=-1)
    e = DEPTH * (spread + e0)
    var = (x - mean).square().mean(dim=-1)
    return e, (var + e0 ** 2) * DEPTH + 2 * e0 * e


def check_corrected(x, eps=1e-5):
    y, mean, rstd = fp8.fp8_layer_norm(x, None, None, eps, fp8.OUT_F32, stats=True)
    x64 = x.cpu().double()
    e, e_var = corrected_errors(x64)
    mean64 = x64.mean(dim=-1)
    d64 = x64 - mean64[:, None]
    var64 = d64.square().mean(dim=-1)
    rstd64 = 1 / torch.sqrt(var64 + eps)
    # the square root's slope: rstd moves by half the variance's relative error
    # (e_var is far below eps here), and rounds three times
    e_rstd = rstd64 * (0.6 * e_var / (var64 + eps) + 4 * U)
    xh64 = d64 * rstd64[:, None]
    err = (e * rstd64)[:, None] + d64.abs() * e_rstd[:, None] + 4 * U * xh64.abs()
    for got, want, tol, what in ((mean, mean64, e + mean64.abs() * U, "mean"), (rstd, rstd64, e_rstd, "rstd"),
                                 (y, xh64, err, "y")):
        off = (got.cpu().double() - want).abs()
        assert bool((off <= tol).all()), f"{what}: {(off / tol).max().item():.3g} of the bound, off by {off.max():.3g}"


@pytest.mark.parametrize("rows,H", SHAPES)
def test_norm_of_rows_around_a_large_mean(rows, H):
    g = torch.Generator().manual_seed(H)
    centre = 500 + 1000 * torch.rand(rows, 1, generator=g)
    x = centre + 0.1 * torch.randn(rows, H, generator=g)
    check_corrected(x.to(device()))
    check_corrected((-3.0 + 0.05 * torch.randn(rows, H, generator=g)).to(BF16).to(device()))


@pytest.mark.parametrize("rows,H", SHAPES)
def test_norm_of_constant_rows(rows, H):
    g = torch.Generator().manual_seed(H + 1)
    for t in (F32, BF16):
        x = (500 + 1000 * torch.rand(rows, 1, generator=g)).expand(rows, H).contiguous().to(t).to(device())
        check_corrected(x)
        _, mean, rstd = fp8.fp8_layer_norm(x, stats=True)
        # what the backward pass makes of these statistics
        assert torch.equal(mean, x[:, 0].float())


def test_norm_of_constant_rows_with_tiny_eps():
    # the variance that the roundings leave must not turn negative
    for H in (96, 1027, 5120, 40001):
        x = torch.full((600, H), 777.7, device=device())
        y, mean, rstd = fp8.fp8_layer_norm(x, None, None, 1e-20, fp8.OUT_F32, stats=True)
        assert bool(torch.isfinite(rstd).all()) and torch.equal(mean, x[:, 0])


def test_norm_of_constant_rows_without_eps():
    # 0 / 0: NaN, or a quotient of what the roundings leave, never an infinity,
    # which an FP8 output would show as its largest value.  With all differences
    # d, |d - off| is within DEPTH d, and a variance d^2 - off^2 above 0 at least
    # 2^-48 d^2 (off^2 has 48 bits): 60 at most
    for H in (7, 96, 300, 1027, 5120, 9001, 20000, 40001):
        x = (500 + 1000 * torch.rand(600, 1, generator=torch.Generator().manual_seed(H))).expand(600, H).contiguous()
        y = fp8.fp8_layer_norm(x.to(device()), None, None, 0.0, fp8.OUT_F32)
        assert not bool(torch.isinf(y).any())
        assert bool((torch.isnan(y) | (y.abs() <= 60)).all())


# ---------------------------------------------------------------------------
# Wide FP32 rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows,H", [(513, 4104), (700, 5120), (900, 6144), (600, 8200), (700, 9001), (520, 12288)])
def test_norm_of_wide_fp32_rows(rows, H):
    # FP32 rows of three groups per thread, with weight and bias of either type
    g = torch.Generator().manual_seed(rows)
    x = (torch.randn(rows, H, generator=g) + 0.3).to(device())
    sy = torch.tensor([0.02], device=device())
    for wt in (BF16, F32):
        w, b = ((k + 0.2 * torch.randn(H, generator=g)).to(wt).to(device()) for k in (1.0, 0.0))
        y64, mean64, rstd64, err = ref.norm(x, w, b, 1e-5)
        for out in (fp8.OUT_BF16, fp8.OUT_F32, fp8.OUT_FP8):
            y, mean, rstd = fp8.fp8_layer_norm(x, w, b, 1e-5, out, sy, stats=True)
            if out == fp8.OUT_FP8:
                ref.check_fp8(y, y64, err, sy, "y")
            else:
                ref.check(y, y64, err, "y")
        e_mean, e_rstd = ref.norm_errors(x.cpu().double(), 1e-5)
        ref.check(mean, mean64, e_mean, "mean")
        ref.check(rstd, rstd64, rstd64 * e_rstd, "rstd")


# ---------------------------------------------------------------------------
# Backward pass: columns past the row's end
# ---------------------------------------------------------------------------

# widths that leave columns of a group, groups of a workgroup, both or none
# behind the row
ENDS = [1, 3, 8, 61, 64, 120, 128, 129, 300, 504, 512, 513, 1000, 1024, 1027, 4096, 5121, 8185, 8192, 8193, 9000, 16383,
        16384, 16390]


@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("H", ENDS)
def test_backward_where_mean_times_rstd_overflows(H, xt, dt):
    # a constant row of 2^80 whose rstd is 2^50: xh is 0 in every column, but
    # -mean * rstd is past FP32's range
    d = device()
    for rows in (1, 3, 40):
        g = torch.Generator().manual_seed(H)
        x = torch.full((rows, H), 2.0 ** 80).to(xt).to(d)
        dy = torch.randn(rows, H, generator=g).to(dt).to(d)
        w = torch.randn(H, generator=g).to(d)
        mean, rstd = torch.full((rows,), 2.0 ** 80, device=d), torch.full((rows,), 2.0 ** 50, device=d)
        dx, dw, db, ex, ew, eb = ref.norm_backward(dy, x, w, mean, rstd, None)
        got = fp8.fp8_layer_norm_backward(dy, x, w, mean, rstd)
        ref.check(got[0], dx, ex, "dx")
        ref.check(got[1], dw, ew, "dweight")
        ref.check(got[2], db, eb, "dbias")


def test_backward_of_a_constant_row_of_its_own_statistics():
    x = torch.full((4, 64), 2.0 ** 121, device=device()).to(BF16)
    _, mean, rstd = fp8.fp8_layer_norm(x, stats=True)
    dy = torch.randn(4, 64, generator=torch.Generator().manual_seed(0)).to(BF16).to(device())
    dx, _, _, ex, _, _ = ref.norm_backward(dy, x, None, mean, rstd, None)
    assert bool(torch.isfinite(dx).all())
    ref.check(fp8.fp8_layer_norm_backward(dy, x, None, mean, rstd)[0], dx, ex, "dx")
