"""GPU: the order of fp8_residual_norm's operations: r = fma(z, f, x) with z =
hidden post_rstd and f = (alpha gate) post_weight, each one FP32 operation, bit for
bit, and what that makes of factors beyond FP32's range.

Inputs of eight bits (BF16 values) and f and z of 24 make z f exact in 64 bits, and
its sum with x too where their exponents lie within four: the value rounded there
once more is the FMA's but where it lies within 2^-53 of a tie."""

import pytest
import torch

import mlp_fp8_quant_amd as fp8

from gpu_util import device

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
# one width for each kernel: 16 lanes a row, a wave, a workgroup, two groups a thread, rows beyond registers
WIDTHS = [100, 500, 4096, 16384, 20000]


def inputs(rows, H, gates, post, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(BF16).to(device())  # noqa: E731
    return (r(rows, H).float(), r(rows, H), r(gates, H) if gates else None, r(H) if post else None)


def factor(alpha, gate, post, rows, H):
    f = torch.full((1, H), alpha, dtype=F32, device=device())
    if gate is not None:
        f = f * gate.float().repeat_interleave(rows // gate.shape[0], dim=0)
    return f if post is None else f * post.float()


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("gates,post", [(0, False), (1, False), (0, True), (3, True)])
def test_stream(gates, post, H):
    x, h, gate, pw = inputs(6, H, gates, post, H + gates)
    _, r, _, post_rstd = fp8.fp8_residual_norm(x, None, h, gate=gate, post_weight=pw, alpha=0.22, stats=True)
    z = h.float() if pw is None else h.float() * post_rstd[:, None]
    f = factor(0.22, gate, pw, 6, H)
    assert torch.equal(r, (z.double() * f.double() + x.double()).float())


@pytest.mark.parametrize("H", [100, 500, 4096, 8192, 9000])
@pytest.mark.parametrize("gates", [0, 1, 3, 3000])
def test_gradient_of_the_block(gates, H):
    # without a post-norm dhidden = dx f, one rounding
    rows = max(6, gates)
    x, h, gate, _ = inputs(rows, H, gates, False, H)
    dr, dy, hid = x, x.flip(0), h.float()
    rstd = torch.ones(rows, device=device())
    dx, dh, *_ = fp8.fp8_residual_norm_backward(dy, x, None, rstd, hid, gate=gate, alpha=0.22, dr=dr)
    assert torch.equal(dh, dx * factor(0.22, gate, None, rows, H))


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("hidden,gate,alpha,want", [(1e-30, 1e38, 100.0, float("inf")), (1e38, 1e-30, 1e-30, 2.0),
                                                    (1e30, 1e30, 1e-30, None)])
def test_factors_beyond_the_range(hidden, gate, alpha, want, H):
    # the factor leaves the range though the product would not; the factor is in it though hidden gate is not
    full = lambda v, *s: torch.full(s, v, dtype=F32, device=device())  # noqa: E731
    x, h, g = full(2.0, 3, H), full(hidden, 3, H), full(gate, H)
    _, r = fp8.fp8_residual_norm(x, None, h, gate=g, alpha=alpha)
    if want is None:
        f = full(alpha, H) * g
        want = (h.double() * f.double() + 2.0).float()
        assert torch.isfinite(want).all() and torch.equal(r, want)
    else:
        assert (r == want).all()
