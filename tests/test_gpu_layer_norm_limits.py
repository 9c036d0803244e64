"""GPU: the layer norm and its backward pass where range and rounding bite:
backward passes whose statistics leave FP32's range in columns past the row's
end.  References are 64-bit, from the formulas."""

import pytest
import torch

import mlp_fp8_quant_amd as fp8
import norm_linear_ref as ref

from gpu_util import device

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


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
