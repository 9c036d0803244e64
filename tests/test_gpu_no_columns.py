"""GPU: norms of rows without a column: no memory is read or written, statistics
are the NaN of 0 / 0, and the backward pass takes them."""

import pytest
import torch

import mlp_fp8_quant_amd as fp8

from gpu_util import device

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def poison(n):
    # what a new tensor of n floats finds in its memory
    torch.full((n,), 7.0, device=device())


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_residual_norm(dtype):
    x, h, w = (torch.empty(s, dtype=dtype, device=device()) for s in ((5, 3, 0), (5, 3, 0), (0,)))
    gate = torch.empty(3, 0, dtype=dtype, device=device())
    poison(15)
    y, r, rstd, post = fp8.fp8_residual_norm(x, w, h, gate=gate, post_weight=w, stats=True)
    assert y.shape == r.shape == x.shape and rstd.shape == post.shape == (5, 3)
    assert rstd.isnan().all() and post.isnan().all()
    got = fp8.fp8_residual_norm_backward(x, r, w, rstd, h, gate=gate, post_weight=w, post_rstd=post)
    assert [t.shape for t in got] == [x.shape, x.shape, (0,), (3, 0), (0,)]
    _, _, rstd, post = fp8.fp8_residual_norm(x, stats=True)
    assert rstd.isnan().all() and post is None
    with pytest.raises(ValueError, match="divide"):
        fp8.fp8_residual_norm(x, w, h, gate=gate.new_empty(4, 0))


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_layer_norm(dtype):
    x, w = torch.empty(5, 0, dtype=dtype, device=device()), torch.empty(0, dtype=dtype, device=device())
    poison(5)
    y, mean, rstd = fp8.fp8_layer_norm(x, w, w, stats=True)
    assert y.shape == x.shape and mean.isnan().all() and rstd.isnan().all() and mean.shape == rstd.shape == (5,)
    dx, dw, db = fp8.fp8_layer_norm_backward(x, x, w, mean, rstd)
    assert dx.shape == x.shape and dw.shape == db.shape == (0,)
