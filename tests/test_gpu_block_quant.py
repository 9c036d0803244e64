"""GPU: codes and scales with a scale for each block of 128, bit for bit
against the oracle's encoder, and SwiGLU that emits them against the 64-bit
formula."""

import pytest
import torch

import block_norm_ref as ref
import mlp_fp8_quant_amd as fp8

from gpu_util import device

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
SHAPES = [(1, 1), (1, 16), (1, 128), (3, 129), (17, 127), (128, 128), (130, 260), (257, 1030), (2, 4096), (300, 8),
          (1000, 33), (129, 4104)]
FORMS = [(False, False), (False, True), (True, False), (True, True)]


def values(M, K, seed, special=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp(4 * torch.randn(M, 1, generator=g))
    if special and M * K > 64:
        x[M // 2] = 0.0                              # rows and columns of zeros, signed
        x[:, K // 2] = -0.0
        x[M // 3, : K // 3] *= 2.0 ** -120           # blocks whose scale is subnormal, or nothing
        x[0, 0] = 3e38
        x[-1, -1] = 1e-45
    return x


def same(x, tile, transpose):
    q, s = fp8.fp8_quant_block(x, tile=tile, transpose=transpose)
    wq, ws = ref.quant(x, tile, transpose)
    assert q.shape == wq.shape and s.shape == ws.shape
    assert torch.equal(s.cpu().view(torch.int32), torch.from_numpy(ws).view(torch.int32)), "scales"
    assert torch.equal(q.cpu(), torch.from_numpy(wq)), "codes"


@pytest.mark.parametrize("tile,transpose", FORMS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,K", SHAPES)
def test_codes_and_scales(M, K, dtype, tile, transpose):
    same(values(M, K, M + K).to(dtype).to(device()), tile, transpose)


@pytest.mark.parametrize("tile,transpose", FORMS)
@pytest.mark.parametrize("odd", [float("nan"), float("inf"), -float("inf")])
def test_nan_and_infinities_stay_in_their_block(odd, tile, transpose):
    x = values(140, 272, 5, special=False)
    x[131, 140] = odd
    clean, cs = fp8.fp8_quant_block(values(140, 272, 5, special=False).to(device()), tile=tile, transpose=transpose)
    q, s = fp8.fp8_quant_block(x.to(device()), tile=tile, transpose=transpose)
    r, c = (140, 131) if transpose else (131, 140)
    bad = torch.zeros(q.shape, dtype=torch.bool)
    bad[r // 128 * 128: r // 128 * 128 + 128, c // 128 * 128: c // 128 * 128 + 128] = True
    if not tile:
        bad[:r] = False
        bad[r + 1:] = False
    assert torch.equal(q.cpu()[~bad], clean.cpu()[~bad])
    at = (r // 128 if tile else r, c // 128)
    assert torch.isnan(s[at]) if odd != odd else torch.isinf(s[at])
    if odd != odd:
        assert (q.cpu()[bad] == 0x7F).all()
    else:
        assert q[r, c] == 0x7F
        bad[r, c] = False
        assert (q.cpu()[bad] & 0x7F == 0).all()


@pytest.mark.parametrize("tile,transpose", FORMS)
def test_given_outputs_and_nothing_past_them(tile, transpose):
    x = values(77, 301, 9).to(BF16).to(device())
    wq, ws = ref.quant(x, tile, transpose)
    codes = torch.full((wq.size + 64,), 0xA5, dtype=torch.uint8, device=device())
    scales = torch.full((ws.size + 16,), -1.0, device=device())
    q, s = fp8.fp8_quant_block(x, tile=tile, transpose=transpose, out=codes[:wq.size].view(wq.shape),
                               scales=scales[:ws.size].view(ws.shape))
    assert q.data_ptr() == codes.data_ptr() and torch.equal(q.cpu(), torch.from_numpy(wq))
    assert (codes[wq.size:] == 0xA5).all() and (scales[ws.size:] == -1).all()


def test_ranks_and_empty_tensors():
    x = values(30, 200, 2).to(BF16).to(device())
    q, s = fp8.fp8_quant_block(x.view(2, 3, 5, 200))
    assert q.shape == (2, 3, 5, 208) and s.shape == (2, 3, 5, 2)
    wq, ws = fp8.fp8_quant_block(x)
    assert torch.equal(q.view(30, 208), wq) and torch.equal(s.view(30, 2), ws)
    q, s = fp8.fp8_quant_block(x[:0])
    assert q.shape == (0, 208) and s.shape == (0, 2)
    q, s = fp8.fp8_quant_block(x[:0], transpose=True)
    assert q.shape == (200, 0) and s.shape == (200, 0)
    q, s = fp8.fp8_quant_block(x[:, :0].contiguous())
    assert q.shape == (30, 0) and s.shape == (30, 0)


@pytest.mark.parametrize("M,K", [(1, 1), (1, 130), (13, 12288), (60, 1000), (257, 128), (1000, 65)])
def test_silu_codes(M, K):
    g = torch.Generator().manual_seed(K)
    a, b = (3 * torch.randn(M, K, generator=g)).to(BF16), torch.randn(M, K, generator=g).to(BF16)
    if M * K > 64:
        a.view(-1)[:6] = torch.tensor([0.0, -0.0, -80.0, 90.0, -200.0, 300.0], dtype=BF16)
        a[M // 2], b[M // 2] = torch.finfo(BF16).min, 1.0      # a masked row: nothing of it is left
    q, s = fp8.silu_mul_2in_block(a.to(device()), b.to(device()))
    v, err = ref.silu_mul(a, b)
    ref.check_codes(q, s, v, err)


def test_silu_of_infinities():
    a = torch.zeros(3, 128, dtype=BF16)
    b = torch.ones(3, 128, dtype=BF16)
    a[0, 5], a[1, 5], a[2, 5] = float("inf"), -float("inf"), float("nan")
    q, s = fp8.silu_mul_2in_block(a.to(device()), b.to(device()))
    assert torch.isinf(s[0, 0]) and torch.isnan(s[1, 0]) and torch.isnan(s[2, 0])   # -Inf / (1 + Inf) is NaN
    assert q[0, 5] == 0x7F and (q[0, :5] == 0).all() and (q[1] == 0x7F).all() and (q[2] == 0x7F).all()


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("transpose", [False, True])
def test_more_elements_than_32_bits_count(tile, transpose):
    # the last rows, 128 of which are a block: as if they were alone
    M, K, last = 256 * 131 + 40, 65537, 128 + 40
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=device())
    x[-last:] = torch.randn(last, K, generator=torch.Generator(device=device()).manual_seed(1), device=device())
    part = x[-last:].clone()
    q, s = fp8.fp8_quant_block(x, tile=tile, transpose=transpose)
    qp, sp = fp8.fp8_quant_block(part, tile=tile, transpose=transpose)
    if transpose:
        assert torch.equal(q[:, M - last:], qp) and torch.equal(s[:, -2:], sp)
        assert not any(bool(c[:, :M - last].any()) for c in q.split(2 ** 13))
    else:
        blocks = 2 if tile else last
        assert torch.equal(q[-last:], qp) and torch.equal(s[-blocks:], sp)
        assert not any(bool(c.any()) for c in q[:-last].split(2 ** 13))


def test_swiglu_of_more_elements_than_32_bits_count():
    M, K, last = 33000, 65536, 50
    g = torch.zeros(M, K, dtype=torch.bfloat16, device=device())
    g[-last:] = torch.randn(last, K, generator=torch.Generator(device=device()).manual_seed(2), device=device())
    u = g + 1
    q, s = fp8.silu_mul_2in_block(g, u)
    qp, sp = fp8.silu_mul_2in_block(g[-last:].clone(), u[-last:].clone())
    assert torch.equal(q[-last:], qp) and torch.equal(s[-last:], sp) and not bool(s[:-last].any())
