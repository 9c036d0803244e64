"""GPU: a dispatch mode sees the tensors that the native front of the binding
allocates, as it sees those of the checks in Python, and the results are the
same."""

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import mlp_fp8_quant_amd as fp8
from mlp_fp8_quant_amd import api

from gpu_util import device

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


class Allocations(TorchDispatchMode):
    """Sizes and types of the tensors made while it is on."""

    def __init__(self):
        super().__init__()
        self.made = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        r = func(*args, **(kwargs or {}))
        if "empty" in func.__name__ or "new_" in func.__name__:
            self.made.append((tuple(r.shape), r.dtype))
        return r


def calls():
    g = torch.Generator().manual_seed(1)
    d = device()
    x = torch.randn(600, 256, generator=g).to(BF16).to(d)
    w = torch.randn(264, 256, generator=g).to(BF16).to(d)
    p = torch.ones(256, device=d)
    one = torch.ones(1, device=d)
    qx, sx = fp8.fp8_quant_block(x)
    qw, sw = fp8.fp8_quant_block(w, tile=True)
    _, mean, rstd = fp8.fp8_layer_norm(x, p, stats=True)
    _, r, rs, prs = fp8.fp8_residual_norm(x, p, x, gate=p, post_weight=p, stats=True)
    return [lambda: fp8.fp8_linear_act(qx, qw, one, one, pre=True),
            lambda: fp8.fp8_linear_act_backward(x, x, fp8.ACT_SILU),
            lambda: fp8.fp8_layer_norm(x, p, stats=True),
            lambda: fp8.fp8_layer_norm_backward(x, x, p, mean, rstd),
            lambda: fp8.fp8_quant_block(x, transpose=True),
            lambda: fp8.silu_mul_2in_block(x, x),
            lambda: fp8.fp8_linear_block(qx, qw, sx, sw, pre=True),
            lambda: fp8.fp8_residual_norm(x, p, x, gate=p, post_weight=p, stats=True),
            lambda: fp8.fp8_residual_norm_backward(x, r, p, rs, x, gate=p, post_weight=p, post_rstd=prs)]


@pytest.mark.parametrize("which", range(9))
def test_a_dispatch_mode_sees_the_results(which, monkeypatch):
    call = calls()[which]
    front = api._load_native()
    assert front is not api._PythonOnly
    plain = call()
    with Allocations() as native:
        got = call()
    monkeypatch.setattr(api, "_native", api._PythonOnly)
    with Allocations() as python:
        call()
    flat = lambda r: [r] if torch.is_tensor(r) else [t for t in r if t is not None]  # noqa: E731
    assert [(tuple(t.shape), t.dtype) for t in flat(got)] == [(tuple(t.shape), t.dtype) for t in flat(plain)]
    for a, b in zip(flat(got), flat(plain)):
        assert torch.equal(a, b)
    for t in flat(got):
        assert (tuple(t.shape), t.dtype) in native.made
    assert sorted(map(str, native.made)) == sorted(map(str, python.made))
