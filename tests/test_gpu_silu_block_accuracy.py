"""GPU: silu(g) u of silu_mul_2in_block within the 9 * 2^-24 of its value that it is
documented to, over every BF16 g.

A block with one value besides zeros has that value / 448 as its scale, one
rounding, so that 448 times the scale gives the value to 10 * 2^-24 (and the
subnormal scale's step, 2^-149)."""

import pytest
import torch

import mlp_fp8_quant_amd as fp8

from gpu_util import device

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("u", [1.0, 1.0078125, 1.1328125, 1.2734375, 1.46875, 1.6328125, 1.8125, 1.9921875, -1.34375,
                               3.0e-3, 1.0e4])
def test_every_g(u):
    g = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).to(device())
    g = g[torch.isfinite(g)]
    a = torch.zeros(g.numel(), 128, dtype=torch.bfloat16, device=device())
    b = torch.zeros_like(a)
    a[:, 5], b[:, 5] = g, u
    assert b[0, 5].item() == torch.tensor(u).to(torch.bfloat16).item()
    _, s = fp8.silu_mul_2in_block(a, b)
    x, y = g.double(), b[0, 5].double()
    v = (x / (1.0 + torch.exp(-x)) * y).abs()
    got = s.view(-1).double() * 448.0
    # (of such g silu(g) is g: the largest values' product with u is beyond FP32, a scale of infinity)
    beyond = v > torch.finfo(torch.float32).max
    assert torch.isinf(got[beyond]).all()
    x, v, got = x[~beyond], v[~beyond], got[~beyond]
    # exp(-g) overflows below g = -88.72, where the value is at most 88.8 e^-88.7 |u|, below 2^-121 |u|
    lost = torch.where(x < -88.7, v, torch.zeros_like(v))
    assert (lost <= y.abs() * 2.0 ** -121).all()
    assert ((got - v).abs() <= v * 10 * U + lost + 448 * 2.0 ** -149).all()
