"""GPU: NaN codes, infinite and far-apart scales on each kernel of
fp8_linear_block: they stay in their rows and columns."""

import pytest
import torch

import block_norm_ref as ref
import mlp_fp8_quant_amd as fp8

from block_tile_shapes import KERNEL_SHAPES
from gpu_util import device
from test_gpu_linear_block import on, operands

pytestmark = pytest.mark.gpu
CASES = [(k, s, w) for k, shapes in KERNEL_SHAPES.items() for s in shapes for w in (False, True)]


@pytest.mark.parametrize("kernel,shape,w_rows", CASES)
def test_nan_codes_and_infinite_scales(kernel, shape, w_rows):
    # in the first, the last and a middle block: the first sums of a tile, its last ones, another batch of scales
    M, N, K = shape
    qx, qw, sx, sw, _ = operands(M, N, K, w_rows, 8)
    clean = fp8.fp8_linear_block(*on(qx, qw, sx, sw), out_kind=fp8.OUT_F32).cpu()
    kb = sx.shape[1]
    row, col = {M - 1, M // 3}, {5, N - 1, N // 2}
    qx[M - 1, 3] = 0x7F
    qx[M // 3, K - 1] = 0xFF
    qw[5, K // 2], qw[N - 1, 0], qw[N // 2, K - 1] = 0x7F, 0xFF, 0x7F
    if M > 8:
        sx[M // 2, kb // 2], sx[1, kb - 1] = float("inf"), float("nan")
        row |= {M // 2, 1}
    at = min(N - 1, 300) // (1 if w_rows else 128)
    sw[at, kb - 1] = float("inf")
    bad_r, bad_c = torch.zeros(M, dtype=torch.bool), torch.zeros(N, dtype=torch.bool)
    bad_r[list(row)], bad_c[list(col)] = True, True
    width = 1 if w_rows else 128
    bad_c[at * width: (at + 1) * width] = True
    y = fp8.fp8_linear_block(*on(qx, qw, sx, sw), out_kind=fp8.OUT_F32).cpu()
    assert torch.equal(y[~bad_r][:, ~bad_c], clean[~bad_r][:, ~bad_c])
    # (a sum of infinities of both signs is NaN, of one infinite; a block's exact zero times an infinity NaN)
    assert not torch.isfinite(y[bad_r]).any() and not torch.isfinite(y[:, bad_c]).any()


@pytest.mark.parametrize("kernel,shape,w_rows", CASES)
def test_scales_far_apart(kernel, shape, w_rows):
    # a block whose scale is 2^60 times the next one's, a row of zero scales, products of scales below the range
    M, N, K = shape
    qx, qw, sx, sw, _ = operands(M, N, K, w_rows, 7)
    sx[:, 0] = 2.0 ** -70
    sx[:, 1] = 2.0 ** -10
    zero = M // 2 if M > 1 else None
    if zero is not None:
        sx[zero] = 0.0
    sw[0, 0] = 2.0 ** -70
    y = fp8.fp8_linear_block(*on(qx, qw, sx, sw), out_kind=fp8.OUT_F32)
    r = torch.tensor(sorted({0, 1, 63, 64, 127, 128, 255, 256, M // 2, M - 1} & set(range(M))))
    y64, _, err, _ = ref.linear(qx[r], qw, sx[r], sw, w_rows)
    ref.check(y[r.to(device())], y64, err)
    assert zero is None or (y[zero] == 0).all()
