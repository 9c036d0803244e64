"""GPU: gelu and its slope as the Linear epilogue evaluates them in FP32, held
relative to their own size in the tail and to their plain form's accuracy.
References are 64-bit, from the formulas."""

import math

import pytest
import torch

import mlp_fp8_quant_amd as fp8
import norm_linear_ref as ref

from gpu_util import device

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
U = ref.U


def gelu_of(z):
    """The kernel's FP32 gelu of FP32 values: an empty sum with z as its bias."""
    q = torch.empty(1, 0, dtype=torch.uint8, device=z.device)
    qw = torch.empty(z.numel(), 0, dtype=torch.uint8, device=z.device)
    s = torch.ones(1, device=z.device)
    return fp8.fp8_linear_act(q, qw, s, s, z, fp8.ACT_GELU, out_kind=fp8.OUT_F32)[0]


def gelu_slope_of(z):
    """The kernel's FP32 slope at BF16 values: the bias's gradient of one row."""
    return fp8.fp8_linear_act_backward(torch.ones_like(z)[None], z[None], fp8.ACT_GELU)[1]


def phi_error(z):
    """Bound of the kernel's error in Phi(z).  With a = |z|, Phi(-a) is a
    polynomial of 1 / (a + c) times 1 / (a + c) times 2^(-a^2 log2(e) / 2): the
    power's argument rounds twice (u a^2 in the power) and its constant is off
    by a quarter of that at most; the power and the reciprocal take a step (2 u)
    each, their products and the polynomial ten half steps at most.  1 - Phi(-a)
    rounds once more."""
    tail = ref.phi(-z.abs())
    return tail * (1.25 * z * z + 14) * U + torch.where(z > 0, ref.phi(z) * U, torch.zeros_like(z))


def test_gelu_keeps_its_relative_accuracy_in_the_tail():
    # down to z = -12.9; below, Phi leaves FP32's normal range
    z = torch.cat([torch.linspace(-12.9, -0.01, 200001), torch.linspace(0.01, 12.9, 50001)]).to(device())
    z64 = z.cpu().double()
    want = z64 * ref.phi(z64)
    err = z64.abs() * phi_error(z64) + 2 * U * want.abs()
    off = (gelu_of(z).cpu().double() - want).abs()
    at = (off / err).argmax()
    assert bool((off <= err).all()), f"at {z64[at]}: {(off / want.abs())[at] / U} half steps"


def test_gelu_slope_keeps_its_accuracy_in_the_tail():
    # every BF16 value between -12.9 and 12.9
    z = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16)
    z = z[(z.float().abs() < 12.9) & (z.float().abs() > 1e-3)].contiguous().to(device())
    z64 = z.cpu().double()
    density = z64 * torch.exp(-z64 * z64 / 2) / math.sqrt(2 * math.pi)
    want = ref.phi(z64) + density
    # the density's factor rounds twice and shares the power's error; the sum rounds once
    err = phi_error(z64) + density.abs() * (1.25 * z64 * z64 + 6) * U + want.abs() * U
    off = (gelu_slope_of(z).cpu().double() - want).abs()
    at = (off / err).argmax()
    assert bool((off <= err).all()), f"at {z64[at]}: off by {off[at]}, bound {err[at]}"


def test_gelu_is_as_exact_as_its_plain_form():
    # root mean square error over random arguments, relative to the values'.
    # The value: at most half a step, that of three roundings that are each
    # anywhere in half a step (u / sqrt 3); the plain form 0.5 z (1 + erf(z /
    # sqrt 2)) has 0.63 of it.  The slope, w or 1 - w: w's power and reciprocal
    # (2 u), three products and the polynomial, together sqrt((4 + 4 + 4) / 3) u
    # of |w| <= 1/2, and the difference's u / sqrt 3: 1.16 u beside slopes of
    # 0.7 in the mean square, 1.6 u
    g = torch.Generator().manual_seed(0)
    z = torch.randn(1 << 20, generator=g).to(device())
    rms = lambda got, want: ((got.cpu().double() - want).square().mean() / want.square().mean()).sqrt().item()  # noqa: E731
    z64 = z.cpu().double()
    plain = 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    own, theirs = rms(gelu_of(z), z64 * ref.phi(z64)), rms(plain, z64 * ref.phi(z64))
    print(f"value {own / U:.3f} u, plain {theirs / U:.3f} u")
    assert own <= U, (own / U, theirs / U)
    zb = (torch.randn(1 << 20, generator=g)).to(BF16).to(device())
    own = rms(gelu_slope_of(zb), ref.act_slope(zb.cpu().double(), fp8.ACT_GELU))
    print(f"slope {own / U:.3f} u")
    assert own <= 1.6 * U, own / U


def test_gelu_of_special_values():
    # as z Phi(z) has them: the sign of a product that underflows, +Inf, and the
    # NaN of -Inf * 0.  (A bias of -0 reaches the activation as +0: z is
    # fma(0, 1, -0), and +0 + -0 = +0)
    inf = float("inf")
    z = torch.tensor([0.0, -0.0, -40.0, -3e38, 40.0, 3.4028234e38, inf, -inf, float("nan"), 2.0 ** -140, -(2.0 ** -140)],
                     device=device())
    y = gelu_of(z).cpu()
    want = torch.tensor([0.0, 0.0, -0.0, -0.0, 40.0, 3.4028234e38, inf, float("nan"), float("nan"), 2.0 ** -141,
                         -(2.0 ** -141)])
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(torch.signbit(y[:7]), torch.signbit(want[:7]))
    assert torch.equal(y[:7], want[:7])
    assert bool(((y[9:].double() - want[9:].double()).abs() <= 2.0 ** -149).all())
    zb = torch.tensor([0.0, -0.0, -40.0, 40.0, -3e38, 3e38], device=device()).to(BF16)
    assert torch.equal(gelu_slope_of(zb).cpu(), torch.tensor([0.5, 0.5, 0.0, 1.0, 0.0, 1.0]))
