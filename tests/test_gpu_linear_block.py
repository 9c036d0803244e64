"""GPU: the FP8 Linear of operands with a scale for each block of 128, against
the 64-bit formula."""

import pytest
import torch

import block_norm_ref as ref
import mlp_fp8_quant_amd as fp8

from gpu_util import device
from norm_linear_ref import ACTS, check_fp8

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def codes(g, rows, K):
    return torch.randint(0, 256, (rows, K), generator=g, dtype=torch.uint8)


def operands(M, N, K, w_rows, seed):
    """Codes of every value but NaN, scales over twelve powers of two."""
    g = torch.Generator().manual_seed(seed)
    fix = lambda q: torch.where(q & 0x7F == 0x7F, q - 1, q)  # noqa: E731
    scale = lambda *s: torch.exp2(12 * torch.rand(*s, generator=g) - 12) * (1 + torch.rand(*s, generator=g))  # noqa: E731
    kb = (K + 127) // 128
    return (fix(codes(g, M, K)), fix(codes(g, N, K)), scale(M, kb), scale(N if w_rows else (N + 127) // 128, kb), g)


def on(*ts):
    return [t.to(device()) if t is not None else None for t in ts]


# sizes that reach every kernel, and both sides of every tile's edges
SHAPES = [(1, 1, 16), (1, 100, 128), (1, 4096, 272), (1, 8192, 400), (7, 20000, 144), (16, 129, 1040), (17, 1, 128),
          (17, 257, 384), (33, 96, 2064), (40, 3001, 256), (64, 130, 512), (65, 2000, 640), (100, 777, 1296),
          (130, 4097, 128), (257, 1023, 272), (600, 900, 528), (513, 2052, 160),
          (20, 9000, 272), (1030, 2100, 400), (700, 3150, 128), (1100, 5003, 272), (2200, 2049, 528), (1024, 3000, 2064),
          (510, 16380, 2064), (60, 18001, 272), (140, 9000, 1296), (500, 4001, 1296), (505, 4002, 1408), (1500, 5003, 528),
          (1500, 1450, 4112)]


@pytest.mark.parametrize("w_rows", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products(M, N, K, w_rows):
    qx, qw, sx, sw, g = operands(M, N, K, w_rows, M + N + K)
    y64, _, err, _ = ref.linear(qx, qw, sx, sw, w_rows)
    d = on(qx, qw, sx, sw)
    y = fp8.fp8_linear_block(*d, out_kind=fp8.OUT_F32)
    ref.check(y, y64, err, "fp32")
    assert torch.equal(y, fp8.fp8_linear_block(*d, out_kind=fp8.OUT_F32))
    assert torch.equal(fp8.fp8_linear_block(*d), y.to(BF16))


@pytest.mark.parametrize("w_rows", [False, True])
def test_workgroups_that_walk_tiles(w_rows):
    # 512 tiles of 256x128 on 256 CUs, ragged on both sides; K ends inside a stage and a batch of scales
    M, N, K = 1020, 16380, 2064
    qx, qw, sx, sw, g = operands(M, N, K, w_rows, 11)
    bias = torch.randn(N, generator=g)
    y = fp8.fp8_linear_block(*on(qx, qw, sx, sw), bias=bias.to(device()), out_kind=fp8.OUT_F32)
    for r in (slice(0, 130), slice(500, 560), slice(960, 1020)):
        y64, _, err, _ = ref.linear(qx[r], qw, sx[r], sw, w_rows, bias)
        ref.check(y[r], y64, err)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N", [(1, 300), (60, 131), (300, 516)])
def test_epilogue(M, N, act):
    K = 272
    qx, qw, sx, sw, g = operands(M, N, K, False, M + act)
    sx, sw = sx * 2.0 ** -8, sw * 2.0 ** -4                    # z of a few units
    for bt, rt in ((None, BF16), (BF16, F32), (F32, None)):
        bias = None if bt is None else torch.randn(N, generator=g).to(bt)
        res = None if rt is None else torch.randn(M, N, generator=g).to(rt)
        y64, z64, err, err_z = ref.linear(qx, qw, sx, sw, False, bias, act, res)
        d, (b, r) = on(qx, qw, sx, sw), on(bias, res)
        y, pre = fp8.fp8_linear_block(*d, bias=b, act=act, residual=r, out_kind=fp8.OUT_F32, pre=True)
        ref.check(y, y64, err, "fp32")
        ref.check(pre, z64, err_z, "pre")
        ref.check(fp8.fp8_linear_block(*d, bias=b, act=act, residual=r), y64, err, "bf16")
        sy = torch.tensor([0.013])
        q = fp8.fp8_linear_block(*d, bias=b, act=act, residual=r, out_kind=fp8.OUT_FP8, sy=sy.to(device()))
        check_fp8(q, y64, err, sy, "fp8")


@pytest.mark.parametrize("M,N", [(1, 64), (50, 200), (300, 700)])
def test_in_place_residual(M, N):
    qx, qw, sx, sw, g = operands(M, N, 400, True, N)
    acc = torch.randn(M, N, generator=g)
    y64, _, err, _ = ref.linear(qx, qw, sx, sw, True, residual=acc)
    got = acc.to(device())
    out = fp8.fp8_linear_block(*on(qx, qw, sx, sw), residual=got, out_kind=fp8.OUT_F32, out=got)
    assert out.data_ptr() == got.data_ptr()
    ref.check(got, y64, err)


@pytest.mark.parametrize("M,N", [(3, 50), (70, 200), (300, 300)])
def test_no_k(M, N):
    e = lambda *s, t=F32: torch.empty(s, dtype=t, device=device())  # noqa: E731
    bias = torch.randn(N, device=device())
    y = fp8.fp8_linear_block(e(M, 0, t=torch.uint8), e(N, 0, t=torch.uint8), e(M, 0), e((N + 127) // 128, 0), bias=bias,
                             out_kind=fp8.OUT_F32)
    assert torch.equal(y, bias.expand(M, N))
    assert fp8.fp8_linear_block(e(0, 32, t=torch.uint8), e(N, 32, t=torch.uint8), e(0, 1), e((N + 127) // 128, 1)).shape == (0, N)


@pytest.mark.parametrize("M,N,K", [(1, 200, 272), (40, 130, 400), (300, 600, 528)])
def test_scales_far_apart(M, N, K):
    # a block whose scale is 2^60 times the next one's, zero scales, products of scales below and above the range
    qx, qw, sx, sw, _ = operands(M, N, K, False, 7)
    sx[:, 0] = 2.0 ** -70
    sx[:, 1] = 2.0 ** -10
    sx[M // 2] = 0.0
    sw[0, 0] = 2.0 ** -70
    y64, _, err, _ = ref.linear(qx, qw, sx, sw, False)
    y = fp8.fp8_linear_block(*on(qx, qw, sx, sw), out_kind=fp8.OUT_F32)
    ref.check(y, y64, err)
    assert (y[M // 2] == 0).all()


@pytest.mark.parametrize("M,N,K", [(1, 200, 272), (40, 130, 400), (300, 600, 528)])
def test_nan_and_infinite_scales_stay_in_their_rows(M, N, K):
    qx, qw, sx, sw, _ = operands(M, N, K, True, 8)
    clean = fp8.fp8_linear_block(*on(qx, qw, sx, sw))
    qx[M - 1, 3], qw[5, K - 1] = 0x7F, 0xFF
    sw[9, 0] = float("inf")
    y = fp8.fp8_linear_block(*on(qx, qw, sx, sw))
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[M - 1], bad[:, 5] = True, True
    assert torch.isnan(y.cpu()[bad]).all()
    assert (~torch.isfinite(y.cpu()[:, 9])).all()
    bad[:, 9] = True
    assert torch.equal(y.cpu()[~bad], clean.cpu()[~bad])


@pytest.mark.parametrize("w_rows", [False, True])
@pytest.mark.parametrize("M,N,K", [(1500, 1450, 1264), (1500, 1450, 1296), (1500, 1450, 1408), (505, 4002, 1264),
                                   (505, 4002, 1296), (505, 4002, 1408), (1500, 1450, 4080), (1500, 1450, 4112)])
def test_infinite_first_scales_stay_in_their_rows(M, N, K, w_rows):
    # even and odd numbers of blocks, the last one whole and not: the two halves of K that a tile's wave groups take
    # end at different blocks
    qx, qw, sx, sw, _ = operands(M, N, K, w_rows, 10)
    y = fp8.fp8_linear_block(*on(qx, qw, sx, sw), out_kind=fp8.OUT_F32)
    sx2, sw2 = sx.clone(), sw.clone()
    sx2[1::2, 0] = float("inf")
    sw2[1::2, 0] = float("nan")
    rows = torch.arange(M) % 2 == 0
    cols = (torch.arange(N) // (1 if w_rows else 128)) % 2 == 0
    y2 = fp8.fp8_linear_block(*on(qx, qw, sx2, sw2), out_kind=fp8.OUT_F32).cpu()
    assert torch.equal(y2[rows][:, cols], y.cpu()[rows][:, cols])
    assert not torch.isfinite(y2[~rows]).any() and y2[:, ~cols].isnan().all()


def test_one_nan_block_of_a_batch_leaves_the_others():
    # what fp8_quant_block makes of a NaN, through the product
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(20, 300, generator=g), torch.randn(50, 300, generator=g)
    q = lambda t, **k: fp8.fp8_quant_block(t.to(BF16).to(device()), **k)  # noqa: E731
    qw, sw = q(w, tile=True)
    qx, sx = q(x)
    clean = fp8.fp8_linear_block(qx, qw, sx, sw)
    x[4, 299] = float("nan")
    qx, sx = q(x)
    y = fp8.fp8_linear_block(qx, qw, sx, sw)
    assert torch.isnan(y[4]).all()
    keep = torch.arange(20) != 4
    assert torch.equal(y.cpu()[keep], clean.cpu()[keep])


def test_leading_dimensions_and_nothing_past_the_output():
    qx, qw, sx, sw, _ = operands(30, 129, 144, False, 3)
    d = on(qx, qw, sx, sw)
    flat = fp8.fp8_linear_block(*d)
    y = fp8.fp8_linear_block(d[0].view(2, 3, 5, 144), d[1], d[2].view(2, 3, 5, 2), d[3])
    assert y.shape == (2, 3, 5, 129) and torch.equal(y.view(30, 129), flat)
    buf = torch.full((30 * 129 + 64,), 7.0, dtype=BF16, device=device())
    fp8.fp8_linear_block(*d, out=buf[:30 * 129].view(30, 129))
    assert torch.equal(buf[:30 * 129].view(30, 129), flat) and (buf[30 * 129:] == 7).all()


def test_most_rows():
    # as many rows as the call takes: more tiles than a launch could number threads for
    M, N, K = 2 ** 31 - 1, 3, 16
    qx, qw, sx, sw, g = operands(64, N, K, False, 5)
    rows = torch.cat((torch.arange(0, 8), torch.randint(8, M - 8, (48,), generator=g), torch.arange(M - 8, M)))
    dqx = torch.zeros(M, K, dtype=torch.uint8, device=device())
    dsx = torch.zeros(M, 1, device=device())
    at = rows.to(device())
    dqx[at], dsx[at] = qx.to(device()), sx.to(device())
    y = fp8.fp8_linear_block(dqx, qw.to(device()), dsx, sw.to(device()))
    y64, _, err, _ = ref.linear(qx, qw, sx, sw, False)
    ref.check(y[at].cpu(), y64, err, "bf16")
    y[at] = 0
    assert not any(bool(part.any()) for part in y.split(2 ** 28))
