"""The libfp8mot calls as PyTorch custom operators (namespace ``fp8mot``).

Pull request "Load static FP8 Cosmos3 Nano/Super checkpoints without
re-quantizing them", first commit message: the two-input SwiGLU carries the
full custom-op contract -- a fake (shape) kernel, opcheck,
torch.compile(fullgraph=True) and graph capture.  Here every hot-path call
is registered with ``torch.library.custom_op``: the real kernel is the
libfp8mot entry point (through ``mlp_fp8_quant_amd.api``), and a fake kernel
states the output shapes and dtypes so that tracing (FakeTensor, dynamo with
fullgraph) never runs the library.  The ops allocate their outputs and
workspaces with torch, launch on the current stream and never synchronize, so
they can be captured in a HIP graph.

Scales are 1-element FP32 device tensors; weights are E4M3 codes (uint8).
"""

import math
from typing import Optional

import torch

from . import api

NS = "fp8mot"


def _rows(t):
    return math.prod(t.shape[:-1])


@torch.library.custom_op(f"{NS}::quant_static", mutates_args=())
def quant_static(x: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    """E4M3 codes of BF16 x at the static per-tensor scale."""
    return api.fp8_quant_static(x, scale)


@quant_static.register_fake
def _(x, scale):
    return torch.empty(x.shape, dtype=torch.uint8, device=x.device)


@torch.library.custom_op(f"{NS}::linear", mutates_args=())
def linear(qx: torch.Tensor, qw: torch.Tensor, sx: torch.Tensor, sw: torch.Tensor,
           accum: int = api.ACC_EXACT) -> torch.Tensor:
    """BF16 y = (qx . qw^T) * (sx * sw)."""
    return api.fp8_linear(qx, qw, sx, sw, accum=accum)


@linear.register_fake
def _(qx, qw, sx, sw, accum=api.ACC_EXACT):
    return torch.empty((*qx.shape[:-1], qw.shape[0]), dtype=torch.bfloat16, device=qx.device)


@torch.library.custom_op(f"{NS}::silu_mul_2in", mutates_args=())
def silu_mul_2in(g: torch.Tensor, u: torch.Tensor, s_out: torch.Tensor,
                 alpha: float = 1.0, beta: float = 0.0) -> torch.Tensor:
    """E4M3 codes of g * sigmoid(alpha g) * (u + beta) at s_out."""
    if alpha == 1.0 and beta == 0.0:
        return api.silu_mul_2in_fp8(g, u, s_out)
    return api.silu_mul_2in_fp8(g, u, s_out, alpha=alpha, beta=beta)


@silu_mul_2in.register_fake
def _(g, u, s_out, alpha=1.0, beta=0.0):
    return torch.empty(g.shape, dtype=torch.uint8, device=g.device)


@torch.library.custom_op(f"{NS}::silu_mul", mutates_args=())
def silu_mul(x: torch.Tensor, s_out: torch.Tensor, alpha: float = 1.0,
             beta: float = 0.0) -> torch.Tensor:
    """One-input SwiGLU-FP8: x [..., 2I] (gate half, then up half) -> [..., I]."""
    return api.silu_mul_fp8(x, s_out, alpha=alpha, beta=beta)


@silu_mul.register_fake
def _(x, s_out, alpha=1.0, beta=0.0):
    return torch.empty((*x.shape[:-1], x.shape[-1] // 2), dtype=torch.uint8, device=x.device)


@torch.library.custom_op(f"{NS}::gated_mlp", mutates_args=())
def gated_mlp(x: torch.Tensor, sx: torch.Tensor, wg: torch.Tensor, sg: torch.Tensor,
              wu: torch.Tensor, su: torch.Tensor, sh: torch.Tensor, wd: torch.Tensor,
              sd: torch.Tensor, accum: int = api.ACC_EXACT) -> torch.Tensor:
    """Static FP8 gated MLP (one quantization of x, fused gate/up + SwiGLU-FP8,
    down projection) -> BF16 [..., H]."""
    return api.gated_mlp_fp8(x, sx, wg, sg, wu, su, sh, wd, sd, accum=accum)


@gated_mlp.register_fake
def _(x, sx, wg, sg, wu, su, sh, wd, sd, accum=api.ACC_EXACT):
    return torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)


@torch.library.custom_op(f"{NS}::qkv", mutates_args=())
def qkv(x: torch.Tensor, sx: torch.Tensor, wq: torch.Tensor, sq: torch.Tensor,
        wk: torch.Tensor, sk: torch.Tensor, wv: torch.Tensor, sv: torch.Tensor,
        accum: int = api.ACC_EXACT) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Split Q/K/V over one shared quantization -> three contiguous BF16 tensors."""
    return api.qkv_fp8(x, sx, wq, sq, wk, sk, wv, sv, accum=accum)


@qkv.register_fake
def _(x, sx, wq, sq, wk, sk, wv, sv, accum=api.ACC_EXACT):
    return tuple(torch.empty((*x.shape[:-1], w.shape[0]), dtype=torch.bfloat16, device=x.device)
                 for w in (wq, wk, wv))


@torch.library.custom_op(f"{NS}::quant_per_row", mutates_args=())
def quant_per_row(x: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """Per-row dynamic quantization -> (codes [..., K], FP32 scales [...])."""
    return api.fp8_quant_per_row(x)


@quant_per_row.register_fake
def _(x):
    return (torch.empty(x.shape, dtype=torch.uint8, device=x.device),
            torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device))


@torch.library.custom_op(f"{NS}::linear_rowwise", mutates_args=())
def linear_rowwise(qx: torch.Tensor, qw: torch.Tensor, sx: torch.Tensor, sw: torch.Tensor,
                   accum: int = api.ACC_EXACT) -> torch.Tensor:
    """BF16 y[m, n] = acc * fp32(sx[m] * sw[n]) (per-token / per-channel scales)."""
    return api.fp8_linear_rowwise(qx, qw, sx, sw, accum=accum)


@linear_rowwise.register_fake
def _(qx, qw, sx, sw, accum=api.ACC_EXACT):
    return torch.empty((*qx.shape[:-1], qw.shape[0]), dtype=torch.bfloat16, device=qx.device)


@torch.library.custom_op(f"{NS}::linear_act", mutates_args=())
def linear_act(qx: torch.Tensor, qw: torch.Tensor, sx: torch.Tensor, sw: torch.Tensor,
               bias: Optional[torch.Tensor] = None, act: int = api.ACT_NONE,
               residual: Optional[torch.Tensor] = None, out_kind: int = api.OUT_BF16,
               sy: Optional[torch.Tensor] = None, rowwise: bool = False,
               accum: int = api.ACC_EXACT) -> torch.Tensor:
    """act((qx . qw^T) * scale + bias) + residual as BF16, FP32 or E4M3 codes."""
    return api.fp8_linear_act(qx, qw, sx, sw, bias, act, residual, out_kind, sy, rowwise,
                              accum=accum)


@linear_act.register_fake
def _(qx, qw, sx, sw, bias=None, act=api.ACT_NONE, residual=None, out_kind=api.OUT_BF16, sy=None,
      rowwise=False, accum=api.ACC_EXACT):
    return torch.empty((*qx.shape[:-1], qw.shape[0]), dtype=api._out_dtype(out_kind),
                       device=qx.device)


@torch.library.custom_op(f"{NS}::linear_act_train", mutates_args=())
def linear_act_train(qx: torch.Tensor, qw: torch.Tensor, sx: torch.Tensor, sw: torch.Tensor,
                     bias: Optional[torch.Tensor] = None, act: int = api.ACT_NONE,
                     residual: Optional[torch.Tensor] = None, out_kind: int = api.OUT_BF16,
                     sy: Optional[torch.Tensor] = None, rowwise: bool = False,
                     accum: int = api.ACC_EXACT) -> tuple[torch.Tensor, torch.Tensor]:
    """linear_act with the activation's argument kept: (y, pre)."""
    return api.fp8_linear_act(qx, qw, sx, sw, bias, act, residual, out_kind, sy, rowwise,
                              pre=True, accum=accum)


@linear_act_train.register_fake
def _(qx, qw, sx, sw, bias=None, act=api.ACT_NONE, residual=None, out_kind=api.OUT_BF16, sy=None,
      rowwise=False, accum=api.ACC_EXACT):
    shape = (*qx.shape[:-1], qw.shape[0])
    return (torch.empty(shape, dtype=api._out_dtype(out_kind), device=qx.device),
            torch.empty(shape, dtype=torch.bfloat16, device=qx.device))


@torch.library.custom_op(f"{NS}::linear_act_backward", mutates_args=())
def linear_act_backward(dy: torch.Tensor, pre: Optional[torch.Tensor],
                        act: int = api.ACT_NONE) -> tuple[torch.Tensor, torch.Tensor]:
    """(dz, dbias) of linear_act's epilogue."""
    return api.fp8_linear_act_backward(dy, pre, act)


@linear_act_backward.register_fake
def _(dy, pre, act=api.ACT_NONE):
    return (torch.empty(dy.shape, dtype=torch.bfloat16, device=dy.device),
            torch.empty(dy.shape[-1], dtype=torch.float32, device=dy.device))


@torch.library.custom_op(f"{NS}::layer_norm", mutates_args=())
def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
               out_kind: int = api.OUT_BF16, sy: Optional[torch.Tensor] = None
               ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Layer norm over the last dimension: (y, mean, rstd)."""
    return api.fp8_layer_norm(x, weight, bias, eps, out_kind, sy, stats=True)


@layer_norm.register_fake
def _(x, weight=None, bias=None, eps=1e-5, out_kind=api.OUT_BF16, sy=None):
    stat = lambda: torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)  # noqa: E731
    return (torch.empty(x.shape, dtype=api._out_dtype(out_kind), device=x.device), stat(), stat())


@torch.library.custom_op(f"{NS}::layer_norm_backward", mutates_args=())
def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor],
                        mean: torch.Tensor, rstd: torch.Tensor,
                        dres: Optional[torch.Tensor] = None
                        ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dx, dweight, dbias) of layer_norm."""
    return api.fp8_layer_norm_backward(dy, x, weight, mean, rstd, dres)


@layer_norm_backward.register_fake
def _(dy, x, weight, mean, rstd, dres=None):
    col = lambda: torch.empty(x.shape[-1], dtype=torch.float32, device=x.device)  # noqa: E731
    return torch.empty(x.shape, dtype=x.dtype, device=x.device), col(), col()


def _like(t, *shape, dtype):
    return torch.empty(shape, dtype=dtype, device=t.device)


def _block_codes(t, lead, cols, lead_scales=None):
    lead_scales = lead if lead_scales is None else lead_scales
    return (_like(t, *lead, api._up(cols, 16), dtype=torch.uint8),
            _like(t, *lead_scales, api._blocks(cols), dtype=torch.float32))


@torch.library.custom_op(f"{NS}::quant_block", mutates_args=())
def quant_block(x: torch.Tensor, tile: bool = False,
                transpose: bool = False) -> tuple[torch.Tensor, torch.Tensor]:
    """(codes, scales) of x with a scale for each block of 128."""
    return api.fp8_quant_block(x, tile, transpose)


@quant_block.register_fake
def _(x, tile=False, transpose=False):
    lead, cols = ((x.shape[1],), x.shape[0]) if transpose else (x.shape[:-1], x.shape[-1])
    return _block_codes(x, lead, cols, (api._blocks(lead[0]),) if tile else None)


@torch.library.custom_op(f"{NS}::silu_mul_block", mutates_args=())
def silu_mul_block(g: torch.Tensor, u: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """(codes, scales) of silu(g) * u with a scale for each 128 columns."""
    return api.silu_mul_2in_block(g, u)


@silu_mul_block.register_fake
def _(g, u):
    return _block_codes(g, g.shape[:-1], g.shape[-1])


@torch.library.custom_op(f"{NS}::linear_block", mutates_args=())
def linear_block(qx: torch.Tensor, qw: torch.Tensor, sx: torch.Tensor, sw: torch.Tensor,
                 bias: Optional[torch.Tensor] = None, act: int = api.ACT_NONE,
                 residual: Optional[torch.Tensor] = None, out_kind: int = api.OUT_BF16,
                 sy: Optional[torch.Tensor] = None) -> torch.Tensor:
    """linear_act of operands with a scale for each block of 128 of K."""
    return api.fp8_linear_block(qx, qw, sx, sw, bias, act, residual, out_kind, sy)


@linear_block.register_fake
def _(qx, qw, sx, sw, bias=None, act=api.ACT_NONE, residual=None, out_kind=api.OUT_BF16, sy=None):
    return _like(qx, *qx.shape[:-1], qw.shape[0], dtype=api._out_dtype(out_kind))


@torch.library.custom_op(f"{NS}::residual_norm", mutates_args=())
def residual_norm(x: torch.Tensor, hidden: torch.Tensor, weight: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, post_weight: Optional[torch.Tensor] = None,
                  alpha: float = 1.0, eps: float = 1e-6, out_kind: int = api.OUT_BF16,
                  sy: Optional[torch.Tensor] = None
                  ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, r, rstd, post_rstd) of a block's output and the stream it is added
    to; post_rstd is empty without post_weight.  (Block codes: residual_norm_block.)"""
    api._out_dtype(out_kind)
    y, r, rstd, post = api.fp8_residual_norm(x, weight, hidden, gate, post_weight, alpha, eps,
                                             out_kind, sy, stats=True)
    return y, r, rstd, rstd.new_empty(0) if post is None else post


@residual_norm.register_fake
def _(x, hidden, weight=None, gate=None, post_weight=None, alpha=1.0, eps=1e-6,
      out_kind=api.OUT_BF16, sy=None):
    stat = _like(x, *x.shape[:-1], dtype=torch.float32)
    return (_like(x, *x.shape, dtype=api._out_dtype(out_kind)), torch.empty_like(x), stat,
            _like(x, 0, dtype=torch.float32) if post_weight is None else torch.empty_like(stat))


@torch.library.custom_op(f"{NS}::residual_norm_block", mutates_args=())
def residual_norm_block(x: torch.Tensor, hidden: torch.Tensor,
                        weight: Optional[torch.Tensor] = None,
                        gate: Optional[torch.Tensor] = None,
                        post_weight: Optional[torch.Tensor] = None, alpha: float = 1.0,
                        eps: float = 1e-6) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(codes, scales, r): residual_norm whose y has a scale for each 128 columns."""
    (q, s), r = api.fp8_residual_norm(x, weight, hidden, gate, post_weight, alpha, eps,
                                      api.OUT_FP8_BLOCK)
    return q, s, r


@residual_norm_block.register_fake
def _(x, hidden, weight=None, gate=None, post_weight=None, alpha=1.0, eps=1e-6):
    return (*_block_codes(x, x.shape[:-1], x.shape[-1]), torch.empty_like(x))


@torch.library.custom_op(f"{NS}::residual_norm_backward", mutates_args=())
def residual_norm_backward(dy: torch.Tensor, r: torch.Tensor, weight: torch.Tensor,
                           rstd: torch.Tensor, hidden: torch.Tensor, gate: torch.Tensor,
                           post_weight: torch.Tensor, post_rstd: torch.Tensor,
                           alpha: float = 1.0, dr: Optional[torch.Tensor] = None
                           ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor,
                                      torch.Tensor]:
    """(dx, dhidden, dweight, dgate, dpost_weight) of residual_norm with all its inputs."""
    return api.fp8_residual_norm_backward(dy, r, weight, rstd, hidden, gate, post_weight, post_rstd,
                                          alpha, dr)


@residual_norm_backward.register_fake
def _(dy, r, weight, rstd, hidden, gate, post_weight, post_rstd, alpha=1.0, dr=None):
    col = lambda t: torch.empty(t.shape, dtype=torch.float32, device=t.device)  # noqa: E731
    return torch.empty_like(r), torch.empty_like(hidden), col(weight), col(gate), col(post_weight)


OPS = (quant_static, linear, silu_mul_2in, silu_mul, gated_mlp, qkv, quant_per_row,
       linear_rowwise, linear_act, linear_act_train, linear_act_backward, layer_norm,
       layer_norm_backward, quant_block, silu_mul_block, linear_block, residual_norm,
       residual_norm_block, residual_norm_backward)
