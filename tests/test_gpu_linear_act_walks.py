"""GPU: FP8 Linears whose workgroups walk from tile to tile, the next tile's first
stages on their way under this tile's epilogue, against 64-bit references."""

import math

import pytest
import torch

import mlp_fp8_quant_amd as fp8
import norm_linear_ref as ref

from gpu_util import device

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
U = ref.U


# (tile, workgroups of it that a CU holds, M, N, K): odd and even numbers of
# 128-K stages above the two that are resident, K a multiple of a stage and
# not, N a multiple of 4 and not
WALKS = [((128, 128), 2, 275, 22001, 784), ((128, 128), 2, 1888, 20152, 384), ((128, 128), 2, 4200, 4304, 1168),
         ((256, 256), 1, 3974, 8185, 656), ((256, 256), 1, 3839, 8664, 1024), ((256, 256), 1, 16244, 1988, 640),
         ((256, 256), 1, 950, 32570, 880),
         ((256, 128), 1, 9944, 1538, 3456), ((256, 128), 1, 1665, 9280, 3936), ((256, 128), 1, 8126, 2945, 2560)]


@pytest.mark.parametrize("tile,per_cu,M,N,K", WALKS, ids=lambda v: str(v))
def test_walked_tiles(tile, per_cu, M, N, K):
    d = device()
    cus = torch.cuda.get_device_properties(d).multi_processor_count
    tiles = math.ceil(M / tile[0]) * math.ceil(N / tile[1])
    assert tiles > per_cu * cus and K > 2 * 128      # a second tile for some workgroup, stages refilled
    act, rowwise = ref.ACTS[(M + N) % 5], M % 2 == 1
    g = torch.Generator(device=d).manual_seed(M)
    rand = lambda r: torch.randint(0, 256, (r, K), generator=g, device=d, dtype=torch.uint8) & 0xBF  # noqa: E731
    qx, qw = (torch.where((q & 0x7F) == 0x7F, torch.zeros_like(q), q) for q in (rand(M), rand(N)))
    scale = lambda n, k: k * (0.5 + torch.rand(n, generator=g, device=d))  # noqa: E731
    sx, sw = scale(M if rowwise else 1, 0.7), scale(N if rowwise else 1, K ** -0.5)
    bias = torch.randn(N, generator=g, device=d)
    res = torch.randn(M, N, generator=g, device=d).to(BF16)
    a, b = (q.view(torch.float8_e4m3fn).double() for q in (qx, qw))
    alpha = (sx[:, None] * sw[None, :]).double()
    bt = b.t().contiguous()
    z64 = (a @ bt) * alpha
    err_z = 1e-5 * alpha * (a.abs() @ bt.abs()) + z64.abs() * U
    z64 += bias.double()
    err_z += z64.abs() * U
    y64 = ref.act(z64, act)
    err = 1.13 * err_z + ref.act_error(z64, act)
    y64 += res.double()
    err += y64.abs() * U
    y, pre = fp8.fp8_linear_act(qx, qw, sx, sw, bias, act, res, fp8.OUT_F32, rowwise=rowwise, pre=True)
    for got, want, e, half in ((y, y64, err, U), (pre, z64, err_z, ref.BF16_HALF)):
        off = (got.double() - want).abs() / (e + (want.abs() + e) * half + 2.0 ** -140)
        assert float(off.max()) <= 1.0, f"worst {float(off.max()):.3g} of the bound, {int((off > 1).sum())} outside"
    assert torch.equal(fp8.fp8_linear_act(qx, qw, sx, sw, bias, act, res, rowwise=rowwise), y.to(BF16))
