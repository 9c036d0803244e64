"""GPU: the epilogue of fp8_linear_block (bias, pre, activation, residual, in
place, each output type) on each of its kernels.

A kernel's sums depend on (M, N, K) only, so its own FP32 product without an
epilogue gives every other call's sums: z = fp32(sum + bias), pre = bf16(z), v =
fp32(act(z) + residual), and y = v, bf16(v) or e4m3(fp32(v * fp32(1 / sy))) follow
bit for bit but for act, whose value is held to its own error.  The product itself
is held to the 64-bit formula on rows of the first, the last and the tiles'
edges."""

import pytest
import torch

import block_norm_ref as ref
import mlp_fp8_quant_amd as fp8

from block_tile_shapes import KERNEL_SHAPES, NO_K
from gpu_util import device
from norm_linear_ref import GELU, GELU_TANH, NONE, RELU, SILU, U, act, act_error
from test_gpu_linear_block import on, operands

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
CASES = [(k, s, w) for k, shapes in KERNEL_SHAPES.items() for s in shapes for w in (False, True)]
# (bias, activation, residual, output, in place)
FORMS = [(BF16, SILU, F32, fp8.OUT_F32, True), (F32, NONE, BF16, fp8.OUT_BF16, True), (None, NONE, F32, fp8.OUT_F32, True),
         (F32, GELU_TANH, None, fp8.OUT_FP8, False), (None, RELU, F32, fp8.OUT_FP8, False),
         (BF16, GELU, BF16, fp8.OUT_F32, False)]


def rows_to_check(M):
    near = {0, 1, 63, 64, 127, 128, 129, 255, 256, 257, 511, 512, M // 2, M - 2, M - 1}
    return torch.tensor(sorted(r for r in near if 0 <= r < M))


@pytest.mark.parametrize("kernel,shape,w_rows", CASES)
def test_epilogue(kernel, shape, w_rows):
    M, N, K = shape
    qx, qw, sx, sw, g = operands(M, N, K, w_rows, M + N + K)
    sx, sw = sx * 2.0 ** -8, sw * 2.0 ** -4                    # z of a few units
    d = on(qx, qw, sx, sw)
    acc = fp8.fp8_linear_block(*d, out_kind=fp8.OUT_F32)
    r = rows_to_check(M)
    y64, _, err, _ = ref.linear(qx[r], qw, sx[r], sw, w_rows)
    ref.check(acc[r.to(device())], y64, err, "product")
    randn = lambda *s: torch.randn(*s, generator=g).to(device())  # noqa: E731
    sy = torch.tensor([0.013], device=device())
    for bt, kind, rt, out, in_place in FORMS:
        bias = None if bt is None else randn(N).to(bt)
        res = None if rt is None else randn(M, N).to(rt)
        z = acc if bias is None else acc + bias.float()
        clean = None if res is None else res.float().clone()   # res may be written over
        to = res if in_place else None
        y, pre = fp8.fp8_linear_block(*d, bias=bias, act=kind, residual=res, out_kind=out, pre=True, out=to,
                                      sy=sy if out == fp8.OUT_FP8 else None)
        assert to is None or y.data_ptr() == res.data_ptr()
        assert torch.equal(pre, z.to(BF16)), "pre"
        if kind == NONE:
            v = z if clean is None else z + clean
        elif kind == RELU:
            v = torch.clamp_min(z, 0.0)
            v = v if clean is None else v + clean
        else:
            # the call's FP32 output, whose rounding the others are
            again = None if clean is None else clean.to(rt)
            v = fp8.fp8_linear_block(*d, bias=bias, act=kind, residual=again, out_kind=fp8.OUT_F32)
            z64 = z.cpu().double()
            # besides its error: sigma(z), exp(-z^2 / 2) below the normal range, 2^-126, are zeros (the hardware's
            # exponential and reciprocal), at most |z| 2^-126 of the product with z
            v64, e = act(z64, kind), act_error(z64, kind) + z64.abs() * 2.0 ** -126
            if clean is not None:
                v64 = v64 + clean.cpu().double()
                e = e + v64.abs() * U
            ref.check(v, v64, e, "act")
        if out == fp8.OUT_FP8:
            want = (v * (1.0 / sy)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            want = v.to(BF16) if out == fp8.OUT_BF16 else v
        assert torch.equal(y, want), (bt, kind, rt, out)


@pytest.mark.parametrize("kernel,shape", [(k, s) for k, shapes in NO_K.items() for s in shapes])
def test_no_k(kernel, shape):
    M, N, _ = shape
    e = lambda *s, t=F32: torch.empty(s, dtype=t, device=device())  # noqa: E731
    args = (e(M, 0, t=torch.uint8), e(N, 0, t=torch.uint8), e(M, 0), e((N + 127) // 128, 0))
    bias, res = torch.randn(N, device=device()), torch.randn(M, N, device=device())
    want = bias + res
    y, pre = fp8.fp8_linear_block(*args, bias=bias, residual=res, out_kind=fp8.OUT_F32, pre=True, out=res)
    assert torch.equal(y, want) and torch.equal(pre, bias.to(BF16).expand(M, N))


@pytest.mark.parametrize("kernel,shape,w_rows", [c for c in CASES if not c[0].startswith("rows")])
def test_nothing_past_the_output(kernel, shape, w_rows):
    M, N, K = shape
    d = on(*operands(M, N, K, w_rows, 1)[:4])
    for kind, t in ((fp8.OUT_BF16, BF16), (fp8.OUT_F32, F32)):
        buf = torch.full((M * N + 4096,), 7.0, dtype=t, device=device())
        pre = torch.full((M * N + 4096,), 7.0, dtype=BF16, device=device())
        fp8.fp8_linear_block(*d, out_kind=kind, out=buf[:M * N].view(M, N), pre=pre[:M * N].view(M, N))
        assert (buf[M * N:] == 7).all() and (pre[M * N:] == 7).all()
        assert not (buf[:M * N] == 7).all()
