"""PyTorch-facing binding of libfp8mot: same names as the C ABI.

Torch provides device memory and the current stream; every computation runs
in libfp8mot's HIP kernels.  Each wrapper checks dtype, device and
contiguity and refuses anything else (a strided tensor is rejected, never
copied), computes outside autograd (results carry no graph, also of inputs
that require gradients: a training loop calls the ``*_backward`` functions
itself), flattens rank-N ``[..., H]`` activations to ``[M, H]``, and maps a
non-OK status to ``Fp8motError``.

Dtypes at this boundary: BF16 tensors are ``torch.bfloat16``; FP8 tensors
are ``torch.uint8`` holding E4M3FN codes; scales are one-element
``torch.float32`` device tensors.
"""

import ctypes
import functools
import math
import warnings

import torch

from . import _lib
from ._lib import Fp8motError  # noqa: F401

OUT_BF16, OUT_FP8, OUT_F32, OUT_FP8_BLOCK = 0, 1, 2, 3
BLOCK = 128   # elements that share a scale in the *_block calls
ACC_EXACT, ACC_FP8_MFMA = 0, 1
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = 0, 1, 2, 3, 4
OBS_MAX, OBS_MOVING_AVG = 0, 1
CONV_E4M3_PACKED, CONV_E4M3_INT, CONV_BF16 = 0, 1, 2
_OUT_DTYPE = {OUT_BF16: torch.bfloat16, OUT_FP8: torch.uint8, OUT_F32: torch.float32}


# Host cost per call matters for the small, latency-bound launches: the raw
# handle of the device's current stream (the capture stream under graph
# capture) is taken without building a Stream object, and pointers go to
# ctypes as plain integers (None for NULL).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(t):
    # the library works on the current HIP device (its CU count and
    # architecture check come from there): tensors on another device are
    # refused rather than launched on a stream of the wrong device
    d = t.get_device()
    if d != _get_device():
        raise ValueError(f"tensors are on cuda:{d} but the current device is "
                         f"cuda:{_get_device()}; call under torch.cuda.device({d})")
    if _raw_stream is not None:
        return _raw_stream(d)
    return torch.cuda.current_stream(t.device).cuda_stream


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _need(t, name, dtype, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (strided tensors are refused)")


def _scale(t, name, device):
    if t is None:
        return None  # the library refuses a NULL scale (dynamic quantization)
    _need(t, name, torch.float32, device)
    if t.numel() != 1:
        raise ValueError(f"{name} must hold exactly one float32")
    return t


def fp8_quant_static(x, scale, out=None):
    """E4M3 codes of BF16 ``x`` at the static per-tensor ``scale``."""
    _need(x, "x", torch.bfloat16)
    _scale(scale, "scale", x.device)
    if out is None:
        out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    _need(out, "out", torch.uint8, x.device)
    if out.numel() != x.numel():
        raise ValueError("out must have as many elements as x")
    _lib.call("fp8_quant_static", _ptr(x), _ptr(out), x.numel(), _ptr(scale),
              _stream(x))
    return out


def fp8_linear(qx, qw, sx, sw, out_kind=OUT_BF16, sy=None, out=None,
               accum=ACC_EXACT):
    """y = (qx . qw^T) * (sx * sw) with qx [..., K] and qw [N, K] E4M3.

    ``accum``: ACC_EXACT (F16 matrix cores on exactly decoded codes, FP32-grade
    accumulation) or ACC_FP8_MFMA (native FP8 matrix cores, 2x the rate, with
    the hardware's 8-product windowed accumulation)."""
    _need(qx, "qx", torch.uint8)
    _need(qw, "qw", torch.uint8, qx.device)
    if qw.dim() != 2 or qx.dim() < 1 or qx.shape[-1] != qw.shape[1]:
        raise ValueError("shapes: qx [..., K], qw [N, K]")
    _scale(sx, "sx", qx.device)
    _scale(sw, "sw", qx.device)
    _scale(sy, "sy", qx.device)
    K = qw.shape[1]
    N = qw.shape[0]
    M = math.prod(qx.shape[:-1])
    if out is None:
        out = torch.empty((*qx.shape[:-1], N), dtype=_OUT_DTYPE[out_kind],
                          device=qx.device)
    _need(out, "out", _OUT_DTYPE[out_kind], qx.device)
    if out.numel() != M * N:
        raise ValueError("out must hold M * N elements")
    _lib.call("fp8_linear", _ptr(qx), _ptr(qw), _ptr(out), M, N, K, _ptr(sx),
              _ptr(sw), out_kind, _ptr(sy), accum, _stream(qx))
    return out


def fp8_quant_per_row(x, out=None, scales=None):
    """Per-row dynamic FP8 quantization of a BF16 [..., K] tensor (K % 16 ==
    0): returns (codes [..., K], FP32 scales [...]) with scale = amax(row) /
    448 and codes = e4m3(x / scale) -- per-token activations, or per-channel
    weights at load."""
    _need(x, "x", torch.bfloat16)
    if x.dim() == 0:
        raise ValueError("x must have a last (K) dimension")
    K = x.shape[-1]
    rows = math.prod(x.shape[:-1])
    if out is None:
        out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _need(out, "out", torch.uint8, x.device)
    _need(scales, "scales", torch.float32, x.device)
    if out.numel() != x.numel() or scales.numel() != rows:
        raise ValueError("out must match x and scales must hold one value per row")
    _lib.call("fp8_quant_per_row", _ptr(x), _ptr(out), _ptr(scales), rows, K,
              _stream(x))
    return out, scales


def fp8_linear_rowwise(qx, qw, sx, sw, out_kind=OUT_BF16, out=None, accum=ACC_EXACT):
    """y[m, n] = acc * fp32(sx[m] * sw[n]) with acc = sum_k dec(qx) dec(qw);
    qx [..., K] E4M3 with per-row scales sx [...] (FP32), qw [N, K] with
    per-channel scales sw [N].  out_kind OUT_BF16 or OUT_F32."""
    _need(qx, "qx", torch.uint8)
    dev = qx.device
    _need(qw, "qw", torch.uint8, dev)
    K = qx.shape[-1]
    N = qw.shape[0]
    if qw.dim() != 2 or qw.shape[1] != K:
        raise ValueError("qw must be [N, K] with qx [..., K]")
    M = math.prod(qx.shape[:-1])
    _need(sx, "sx", torch.float32, dev)
    _need(sw, "sw", torch.float32, dev)
    if sx.numel() != M or sw.numel() != N:
        raise ValueError("sx must hold one scale per row of qx and sw one per row of qw")
    dtype = {OUT_BF16: torch.bfloat16, OUT_F32: torch.float32}.get(out_kind)
    if dtype is None:
        raise ValueError("out_kind must be OUT_BF16 or OUT_F32")
    if out is None:
        out = torch.empty((*qx.shape[:-1], N), dtype=dtype, device=dev)
    _need(out, "out", dtype, dev)
    if out.numel() != M * N:
        raise ValueError("out must hold M * N elements")
    _lib.call("fp8_linear_rowwise", _ptr(qx), _ptr(qw), _ptr(out), M, N, K,
              _ptr(sx), _ptr(sw), out_kind, accum, _stream(qx))
    return out


# The calls below take many tensors and are made once per token or training
# step.  Their common case -- plain contiguous tensors that fit, on
# the current device -- is marshalled natively (csrc/binding.cpp), which
# returns None for anything else and the status where the library refuses;
# what follows the native call is every check and its message, and all there
# is where the native front is not built (about 5 us more a call).
_native = None
NO_FRONT = ("the native front of the binding is missing or does not load: fp8_linear_act, fp8_layer_norm, the calls "
            "with a scale for each block, fp8_residual_norm and the backward passes take longer on the host (build it "
            "with `python -m mlp_fp8_quant_amd.build`)")


class _PythonOnly:
    linear_act = linear_act_backward = layer_norm = layer_norm_backward = quant_block = silu_mul_block = \
        linear_block = residual_norm = residual_norm_backward = staticmethod(lambda *args: None)


def _load_native():
    global _native
    try:
        from . import _binding
        _native = _binding
    except ImportError:
        warnings.warn(NO_FRONT)
        _native = _PythonOnly
    return _native


_Tensor = torch.Tensor
_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8


def _fit(t, name, dtype, dev, n=None, what=None):
    if not (type(t) is _Tensor and t.dtype is dtype and t.get_device() == dev and t.is_contiguous()):
        _need(t, name, dtype, torch.device("cuda", dev))
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} must hold {what}")


def _fit_float(t, name, dev, n, what, dtype=None):
    """A BF16 or FP32 tensor of n elements (``dtype`` where only one of the
    types fits), or None; returns its FP8MOT_ELEM code (0 for None)."""
    if t is None:
        return 0
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    d = t.dtype
    if (d is not _BF16 and d is not _F32) or (dtype is not None and d is not dtype):
        raise ValueError(f"{name} must be {dtype or 'torch.bfloat16 or torch.float32'}, got {d}")
    _fit(t, name, d, dev, n, what)
    return 1 if d is _F32 else 0


def _on_gpu(t, name, dtype=None):
    """The device index of a call's first tensor, checked by itself."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is None and t.dtype is not _BF16 and t.dtype is not _F32:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    dev = t.get_device()
    if dev < 0 or not t.is_contiguous() or (dtype is not None and t.dtype is not dtype):
        _need(t, name, dtype or t.dtype)
    if t.dim() == 0:
        raise ValueError(f"{name} must have a last dimension")
    return dev


def _out_dtype(out_kind):
    dtype = _OUT_DTYPE.get(out_kind)
    if dtype is None:
        raise ValueError("out_kind must be OUT_BF16, OUT_FP8 or OUT_F32")
    return dtype


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(func, *sizes):
    # a pure function of the sizes
    return int(getattr(_lib.lib(), func)(*sizes))


def _scratch(func, sizes, t, ws):
    """(pointer, bytes) of a call's workspace: the caller's, a new one, or
    none where the sizes need none."""
    if ws is None:
        nb = _workspace_bytes(func, *sizes)
        if nb == 0:
            return None, None, 0
        ws = t.new_empty(nb, dtype=_U8)
    else:
        _fit(ws, "workspace", _U8, t.get_device())
    return ws, ws.data_ptr(), ws.numel()


def fp8_linear_act_workspace(M, N, K):
    return _workspace_bytes("fp8_linear_act_workspace", M, N, K)


def fp8_linear_act(qx, qw, sx, sw, bias=None, act=ACT_NONE, residual=None, out_kind=OUT_BF16,
                   sy=None, rowwise=False, pre=False, out=None, accum=ACC_EXACT, workspace=None):
    """y = act((qx . qw^T) * scale + bias) + residual in one pass, with
    qx [..., K] and qw [N, K] E4M3 and y [..., N] BF16, FP32 or (at the scale
    ``sy``) E4M3 codes.

    ``act``: ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH or ACT_SILU.  ``bias``
    [N] and ``residual`` [..., N] are BF16 or FP32; ``out`` may be the residual
    itself where the types agree.  ``rowwise``: sx holds one scale per row of
    qx and sw one per row of qw (as fp8_linear_rowwise); else one scale each.
    ``pre``: True, or a BF16 tensor [..., N], keeps the activation's argument
    for fp8_linear_act_backward and makes the call return (y, pre)."""
    r = (_native or _load_native()).linear_act(qx, qw, sx, sw, bias, act, residual, out_kind, sy,
                                               rowwise, pre, out, accum, workspace)
    if r is not None:
        return r if type(r) is not int else _lib.fail("fp8_linear_act", r)
    dev = _on_gpu(qx, "qx", _U8)
    _fit(qw, "qw", _U8, dev)
    shape = qx.shape
    if qw.dim() != 2 or shape[-1] != qw.shape[1]:
        raise ValueError("shapes: qx [..., K], qw [N, K]")
    N, K = qw.shape
    M = qx.numel() // K if K else math.prod(shape[:-1])
    if rowwise:
        _fit(sx, "sx", _F32, dev, M, "one scale per row of qx")
        _fit(sw, "sw", _F32, dev, N, "one scale per row of qw")
    else:
        if sx is not None:   # the library refuses a NULL scale (dynamic quantization)
            _fit(sx, "sx", _F32, dev, 1, "exactly one float32")
        if sw is not None:
            _fit(sw, "sw", _F32, dev, 1, "exactly one float32")
    dtype = _out_dtype(out_kind)
    sy_ptr = None
    if out_kind == OUT_FP8 and sy is not None:
        _fit(sy, "sy", _F32, dev, 1, "exactly one float32")
        sy_ptr = sy.data_ptr()
    bias_elem = _fit_float(bias, "bias", dev, N, "N elements")
    res_elem = _fit_float(residual, "residual", dev, M * N, "M * N elements")
    out_shape = (*shape[:-1], N)
    if out is None:
        out = qx.new_empty(out_shape, dtype=dtype)
    else:
        _fit(out, "out", dtype, dev, M * N, "M * N elements")
    keep = None
    if pre is not False and pre is not None:
        if pre is True:
            keep = qx.new_empty(out_shape, dtype=_BF16)
        else:
            keep = pre
            _fit(keep, "pre", _BF16, dev, M * N, "M * N elements")
    _ws, ws_ptr, ws_bytes = _scratch("fp8_linear_act_workspace", (M, N, K), qx, workspace)
    _lib.call("fp8_linear_act", qx.data_ptr(), qw.data_ptr(), out.data_ptr(), M, N, K, _ptr(sx), _ptr(sw),
              1 if rowwise else 0, _ptr(bias), bias_elem, act, _ptr(residual), res_elem, _ptr(keep),
              out_kind, sy_ptr, accum, ws_ptr, ws_bytes, _stream(qx))
    return out if keep is None else (out, keep)


def fp8_linear_act_backward_workspace(M, N):
    return _workspace_bytes("fp8_linear_act_backward_workspace", M, N)


def fp8_linear_act_backward(dy, pre, act=ACT_NONE, dz=None, dbias=None, workspace=None):
    """Backward pass of fp8_linear_act's epilogue: (dz, dbias) with
    dz = dy * act'(pre) (BF16, shaped as dy [..., N]) and dbias its sum over
    rows (FP32 [N], summed before the rounding of dz).  ``pre`` is what
    fp8_linear_act kept (None allowed for ACT_NONE); ``dz`` may be dy or pre
    itself."""
    r = (_native or _load_native()).linear_act_backward(dy, pre, act, dz, dbias, workspace)
    if r is not None:
        return r if type(r) is not int else _lib.fail("fp8_linear_act_backward", r)
    dev = _on_gpu(dy, "dy", _BF16)
    n = dy.numel()
    N = dy.shape[-1]
    M = n // N if N else 0
    if pre is not None:
        _fit(pre, "pre", _BF16, dev, n, "as many elements as dy")
    if dz is None:
        dz = torch.empty_like(dy)
    else:
        _fit(dz, "dz", _BF16, dev, n, "as many elements as dy")
    if dbias is None:
        dbias = dy.new_empty(N, dtype=_F32)
    else:
        _fit(dbias, "dbias", _F32, dev, N, "N elements")
    _ws, ws_ptr, ws_bytes = _scratch("fp8_linear_act_backward_workspace", (M, N), dy, workspace)
    _lib.call("fp8_linear_act_backward", dy.data_ptr(), _ptr(pre), act, dz.data_ptr(), dbias.data_ptr(), M, N,
              ws_ptr, ws_bytes, _stream(dy))
    return dz, dbias


def _nothing(*stats):
    """The statistics of rows without a column, which the library leaves as they are: 0 / 0."""
    for t in stats:
        if t is not None:
            t.fill_(math.nan)


def fp8_layer_norm(x, weight=None, bias=None, eps=1e-5, out_kind=OUT_BF16, sy=None, stats=False,
                   out=None):
    """Layer norm over the last dimension of x [..., H] (BF16 or FP32):
    y = (x - mean) * rstd * weight + bias as BF16, FP32 or (at the scale
    ``sy``) E4M3 codes for the Linears that read it.  weight and bias [H]:
    both BF16 or both FP32, or None.  ``stats`` makes the call return
    (y, mean, rstd), FP32 [...], for fp8_layer_norm_backward.  ``out`` may be
    x itself where the types agree."""
    r = (_native or _load_native()).layer_norm(x, weight, bias, eps, out_kind, sy, stats, out)
    if r is not None:
        return r if type(r) is not int else _lib.fail("fp8_layer_norm", r)
    dev = _on_gpu(x, "x")
    xt = x.dtype
    n = x.numel()
    H = x.shape[-1]
    rows = n // H if H else math.prod(x.shape[:-1])
    wb_elem = _fit_float(weight, "weight", dev, H, "H elements")
    b_elem = _fit_float(bias, "bias", dev, H, "H elements", None if weight is None else weight.dtype)
    dtype = _out_dtype(out_kind)
    sy_ptr = None
    if out_kind == OUT_FP8 and sy is not None:
        _fit(sy, "sy", _F32, dev, 1, "exactly one float32")
        sy_ptr = sy.data_ptr()
    if out is None:
        out = torch.empty_like(x) if dtype is xt else x.new_empty(x.shape, dtype=dtype)
    else:
        _fit(out, "out", dtype, dev, n, "as many elements as x")
    mean = rstd = None
    if stats:
        mean = x.new_empty(x.shape[:-1], dtype=_F32)
        rstd = torch.empty_like(mean)
        if not H:
            _nothing(mean, rstd)
    _lib.call("fp8_layer_norm", x.data_ptr(), 1 if xt is _F32 else 0, _ptr(weight), _ptr(bias),
              wb_elem if weight is not None else b_elem, out.data_ptr(), out_kind, sy_ptr, _ptr(mean),
              _ptr(rstd), rows, H, eps, _stream(x))
    return (out, mean, rstd) if stats else out


def fp8_layer_norm_backward_workspace(rows, H):
    return _workspace_bytes("fp8_layer_norm_backward_workspace", rows, H)


def fp8_layer_norm_backward(dy, x, weight, mean, rstd, dres=None, dx=None, dweight=None,
                            dbias=None, workspace=None):
    """Backward pass of fp8_layer_norm: (dx, dweight, dbias) for the gradient
    dy [..., H] (BF16 or FP32) of its output.  mean and rstd are what
    fp8_layer_norm(stats=True) returned; ``dres`` (x's type) is the gradient
    that reaches x past the norm and is added to dx before its rounding; dx
    has x's type, dweight and dbias are FP32 [H]."""
    r = (_native or _load_native()).layer_norm_backward(dy, x, weight, mean, rstd, dres, dx,
                                                        dweight, dbias, workspace)
    if r is not None:
        return r if type(r) is not int else _lib.fail("fp8_layer_norm_backward", r)
    dev = _on_gpu(x, "x")
    xt = x.dtype
    n = x.numel()
    H = x.shape[-1]
    rows = n // H if H else math.prod(x.shape[:-1])
    if dy is None:
        raise ValueError("dy must be a tensor")
    dy_elem = _fit_float(dy, "dy", dev, n, "as many elements as x")
    w_elem = _fit_float(weight, "weight", dev, H, "H elements")
    _fit_float(dres, "dres", dev, n, "as many elements as x", xt)
    _fit(mean, "mean", _F32, dev, rows, "one value per row")
    _fit(rstd, "rstd", _F32, dev, rows, "one value per row")
    if dx is None:
        dx = torch.empty_like(x)
    else:
        _fit(dx, "dx", xt, dev, n, "as many elements as x")
    if dweight is None:
        dweight = x.new_empty(H, dtype=_F32)
    else:
        _fit(dweight, "dweight", _F32, dev, H, "H elements")
    if dbias is None:
        dbias = torch.empty_like(dweight)
    else:
        _fit(dbias, "dbias", _F32, dev, H, "H elements")
    _ws, ws_ptr, ws_bytes = _scratch("fp8_layer_norm_backward_workspace", (rows, H), x, workspace)
    _lib.call("fp8_layer_norm_backward", dy.data_ptr(), dy_elem, x.data_ptr(), 1 if xt is _F32 else 0, _ptr(weight),
              w_elem, mean.data_ptr(), rstd.data_ptr(), _ptr(dres), dx.data_ptr(), dweight.data_ptr(),
              dbias.data_ptr(), rows, H, ws_ptr, ws_bytes, _stream(x))
    return dx, dweight, dbias


def _up(n, to):
    return (n + to - 1) // to * to


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _codes(like, lead, cols, out, scales, lead_scales=None):
    """Codes [*lead, cols up to a multiple of 16] and scales [*lead_scales, blocks of cols]
    of a block-scaled result: the caller's or new ones."""
    dev = like.get_device()
    shape, sshape = (*lead, _up(cols, 16)), (*(lead if lead_scales is None else lead_scales), _blocks(cols))
    if out is None:
        out = like.new_empty(shape, dtype=_U8)
    else:
        _fit(out, "out", _U8, dev, math.prod(shape), "rows of codes padded to a multiple of 16")
    if scales is None:
        scales = like.new_empty(sshape, dtype=_F32)
    else:
        _fit(scales, "scales", _F32, dev, math.prod(sshape), "one scale per block of 128")
    return out, scales


def fp8_quant_block(x, tile=False, transpose=False, out=None, scales=None):
    """E4M3 codes of x [..., K] (BF16 or FP32) with an FP32 scale, amax / 448,
    for each block of 128 columns of a row -- or, ``tile``, for each 128 x 128
    tile of a 2-D x.  ``transpose``: of the transposed x [M, K], whose rows then
    are x's columns (a product's backward pass needs them).  Returns (codes,
    scales): codes [..., ld(K)] and scales [..., nb(K)], transposed [K, ld(M)]
    and [K, nb(M)], tiles [nb(rows), nb(columns)], with nb(n) = ceil(n / 128) and
    ld(n) = n up to a multiple of 16; the codes past n are zeros', so that
    fp8_linear_block takes them as they are."""
    r = (_native or _load_native()).quant_block(x, tile, transpose, out, scales)
    if r is not None:
        return r if type(r) is not int else _lib.fail("fp8_quant_block", r)
    dev = _on_gpu(x, "x")
    if (tile or transpose) and x.dim() != 2:
        raise ValueError("x must be 2-D for tiles and for the transposed codes")
    K = x.shape[-1]
    M = math.prod(x.shape[:-1])
    lead, cols = ((K,), M) if transpose else (x.shape[:-1], K)
    out, scales = _codes(x, lead, cols, out, scales, (_blocks(lead[0]),) if tile else None)
    _lib.call("fp8_quant_block", x.data_ptr(), 1 if x.dtype is _F32 else 0, out.data_ptr(), scales.data_ptr(), M, K,
              1 if tile else 0, 1 if transpose else 0, _stream(x))
    return out, scales


def silu_mul_2in_block(g, u, out=None, scales=None):
    """silu(g) * u of two BF16 tensors [..., K] as E4M3 codes with an FP32 scale
    for each 128 columns: (codes [..., ld(K)], scales [..., nb(K)]), see
    fp8_quant_block."""
    r = (_native or _load_native()).silu_mul_block(g, u, out, scales)
    if r is not None:
        return r if type(r) is not int else _lib.fail("silu_mul_2in_block", r)
    dev = _on_gpu(g, "g", _BF16)
    _fit(u, "u", _BF16, dev)
    if g.shape != u.shape:
        raise ValueError("g and u must have the same shape")
    K = g.shape[-1]
    out, scales = _codes(g, g.shape[:-1], K, out, scales)
    _lib.call("silu_mul_2in_block", g.data_ptr(), u.data_ptr(), out.data_ptr(), scales.data_ptr(),
              math.prod(g.shape[:-1]), K, _stream(g))
    return out, scales


def fp8_linear_block(qx, qw, sx, sw, bias=None, act=ACT_NONE, residual=None, out_kind=OUT_BF16, sy=None, pre=False,
                     out=None):
    """fp8_linear_act for operands with a scale for each block of 128 of K:
    qx [..., K] and qw [N, K] E4M3 (K a multiple of 16, as fp8_quant_block pads
    it), sx [..., nb(K)], and sw [nb(N), nb(K)] for 128 x 128 tiles of a weight or
    [N, nb(K)] for its rows (a weight's gradient: dy's and x's transposed codes).
    bias, act, residual, out_kind, sy, pre and out as there; no workspace."""
    r = (_native or _load_native()).linear_block(qx, qw, sx, sw, bias, act, residual, out_kind, sy, pre, out)
    if r is not None:
        return r if type(r) is not int else _lib.fail("fp8_linear_block", r)
    dev = _on_gpu(qx, "qx", _U8)
    _fit(qw, "qw", _U8, dev)
    shape = qx.shape
    if qw.dim() != 2 or shape[-1] != qw.shape[1]:
        raise ValueError("shapes: qx [..., K], qw [N, K]")
    N, K = qw.shape
    M = math.prod(shape[:-1])
    kb = _blocks(K)
    _fit(sx, "sx", _F32, dev, M * kb, "one scale per row and block of 128 of qx")
    _fit(sw, "sw", _F32, dev)
    if sw.numel() not in (N * kb, _blocks(N) * kb):
        raise ValueError("sw must hold one scale per row (or 128 rows) and block of 128 of qw")
    w_rows = sw.numel() != _blocks(N) * kb
    dtype = _out_dtype(out_kind)
    sy_ptr = None
    if out_kind == OUT_FP8 and sy is not None:
        _fit(sy, "sy", _F32, dev, 1, "exactly one float32")
        sy_ptr = sy.data_ptr()
    bias_elem = _fit_float(bias, "bias", dev, N, "N elements")
    res_elem = _fit_float(residual, "residual", dev, M * N, "M * N elements")
    out_shape = (*shape[:-1], N)
    if out is None:
        out = qx.new_empty(out_shape, dtype=dtype)
    else:
        _fit(out, "out", dtype, dev, M * N, "M * N elements")
    keep = None
    if pre is not False and pre is not None:
        if pre is True:
            keep = qx.new_empty(out_shape, dtype=_BF16)
        else:
            keep = pre
            _fit(keep, "pre", _BF16, dev, M * N, "M * N elements")
    _lib.call("fp8_linear_block", qx.data_ptr(), qw.data_ptr(), out.data_ptr(), M, N, K, sx.data_ptr(), sw.data_ptr(),
              1 if w_rows else 0, _ptr(bias), bias_elem, act, _ptr(residual), res_elem, _ptr(keep), out_kind, sy_ptr,
              _stream(qx))
    return out if keep is None else (out, keep)


def _gates(gate, dev, rows, H):
    """(number of gates, FP8MOT_ELEM code) of gate [H] or [gates, H]."""
    if gate is None:
        return 1, 0
    elem = _fit_float(gate, "gate", dev, None, None)
    if gate.dim() not in (1, 2) or gate.shape[-1] != H:
        raise ValueError("gate must be [H] or [gates, H]")
    gates = gate.shape[0] if gate.dim() == 2 else 1
    if gates < 1 or rows % gates:
        raise ValueError("the number of gates must divide the number of rows")
    return gates, elem


def fp8_residual_norm(x, weight=None, hidden=None, gate=None, post_weight=None, alpha=1.0, eps=1e-6,
                      out_kind=OUT_BF16, sy=None, stats=False, out=None, stream_out=None):
    """What stands between two blocks, in one pass over x and hidden [..., H]
    (BF16 or FP32 each): the root-mean-square norm of the block's output hidden
    (with ``post_weight``), its gate, the residual addition and the norm before
    the next block:

        v = hidden * rsqrt(mean(hidden^2) + eps) * post_weight    (or hidden)
        r = x + alpha * gate * v
        y = r * rsqrt(mean(r^2) + eps) * weight

    with alpha * gate * post_weight formed first, as one FP32 factor of hidden's
    norm.  ``gate`` [H], or [gates, H] with a gate for each rows / gates rows.  Returns
    (y, r): y BF16, FP32 or (at the scale ``sy``) E4M3 codes, or with
    OUT_FP8_BLOCK a pair (codes, scales) as fp8_quant_block gives; r has x's type
    and is written to ``stream_out`` (which may be x itself) where that is given.
    ``stats``: (y, r, rstd, post_rstd), FP32 [...] for the backward pass.
    Without ``hidden`` it is the norm of x alone, and r None."""
    if hidden is None and (gate is not None or post_weight is not None or stream_out is not None):
        raise ValueError("gate, post_weight and stream_out go with hidden")
    r = (_native or _load_native()).residual_norm(x, weight, hidden, gate, post_weight, alpha, eps, out_kind, sy, stats,
                                                  out, stream_out)
    if r is not None:
        return r if type(r) is not int else _lib.fail("fp8_residual_norm", r)
    dev = _on_gpu(x, "x")
    xt = x.dtype
    n, H = x.numel(), x.shape[-1]
    rows = n // H if H else math.prod(x.shape[:-1])
    h_elem = _fit_float(hidden, "hidden", dev, n, "as many elements as x")
    w_elem = _fit_float(weight, "weight", dev, H, "H elements")
    p_elem = _fit_float(post_weight, "post_weight", dev, H, "H elements", None if weight is None else weight.dtype)
    gates, g_elem = _gates(gate, dev, rows, H)
    scales = sy_ptr = None
    if out_kind == OUT_FP8_BLOCK:
        out, scales = _codes(x, x.shape[:-1], H, *((None, None) if out is None else out))
    else:
        dtype = _out_dtype(out_kind)
        if out_kind == OUT_FP8 and sy is not None:
            _fit(sy, "sy", _F32, dev, 1, "exactly one float32")
            sy_ptr = sy.data_ptr()
        if out is None:
            out = x.new_empty(x.shape, dtype=dtype)
        else:
            _fit(out, "out", dtype, dev, n, "as many elements as x")
    if hidden is not None:
        if stream_out is None:
            stream_out = torch.empty_like(x)
        else:
            _fit(stream_out, "stream_out", xt, dev, n, "as many elements as x")
    rstd = post_rstd = None
    if stats:
        rstd = x.new_empty(x.shape[:-1], dtype=_F32)
        if post_weight is not None:
            post_rstd = torch.empty_like(rstd)
        if not H:
            _nothing(rstd, post_rstd)
    _lib.call("fp8_residual_norm", x.data_ptr(), 1 if xt is _F32 else 0, _ptr(hidden), h_elem, _ptr(gate), g_elem,
              gates, _ptr(post_weight), _ptr(weight), w_elem if weight is not None else p_elem, _ptr(stream_out),
              out.data_ptr(), out_kind, sy_ptr, _ptr(scales), _ptr(rstd), _ptr(post_rstd), rows, H, alpha, eps,
              _stream(x))
    y = out if scales is None else (out, scales)
    return (y, stream_out, rstd, post_rstd) if stats else (y, stream_out)


def fp8_residual_norm_backward_workspace(rows, H, gates=1):
    return _workspace_bytes("fp8_residual_norm_backward_workspace", rows, H, gates)


def fp8_residual_norm_backward(dy, r, weight, rstd, hidden=None, gate=None, post_weight=None, post_rstd=None, alpha=1.0,
                               dr=None, dx=None, dhidden=None, dweight=None, dgate=None, dpost_weight=None,
                               workspace=None):
    """Backward pass of fp8_residual_norm: (dx, dhidden, dweight, dgate,
    dpost_weight) for the gradients dy [..., H] of y and ``dr`` (r's type) of r.
    r, rstd and post_rstd are what the forward pass returned with ``stats``
    (r is x where there was no hidden).  dx has r's type, dhidden hidden's, which
    dy has to have too; dweight and dpost_weight are FP32 [H], dgate FP32 shaped
    as gate.  What has no input (dhidden without hidden, ...) is None."""
    if hidden is None and (gate is not None or post_weight is not None):
        raise ValueError("gate and post_weight go with hidden")
    res = (_native or _load_native()).residual_norm_backward(dy, r, weight, rstd, hidden, gate, post_weight, post_rstd,
                                                             alpha, dr, dx, dhidden, dweight, dgate, dpost_weight,
                                                             workspace)
    if res is not None:
        return res if type(res) is not int else _lib.fail("fp8_residual_norm_backward", res)
    dev = _on_gpu(r, "r")
    rt = r.dtype
    n, H = r.numel(), r.shape[-1]
    rows = n // H if H else math.prod(r.shape[:-1])
    if dy is None:
        raise ValueError("dy must be a tensor")
    h_elem = _fit_float(dy, "dy", dev, n, "as many elements as r")
    _fit_float(hidden, "hidden", dev, n, "as many elements as r", dy.dtype)
    w_elem = _fit_float(weight, "weight", dev, H, "H elements")
    p_elem = _fit_float(post_weight, "post_weight", dev, H, "H elements", None if weight is None else weight.dtype)
    gates, g_elem = _gates(gate, dev, rows, H)
    _fit_float(dr, "dr", dev, n, "as many elements as r", rt)
    _fit(rstd, "rstd", _F32, dev, rows, "one value per row")
    if post_weight is not None:
        _fit(post_rstd, "post_rstd", _F32, dev, rows, "one value per row")

    def made(t, name, there, shape, dtype, what):
        if not there:
            if t is not None:
                raise ValueError(f"{name} has no input whose gradient it could be")
            return None
        if t is None:
            return r.new_empty(shape, dtype=dtype)
        _fit(t, name, dtype, dev, math.prod(shape), what)
        return t

    dx = made(dx, "dx", True, r.shape, rt, "as many elements as r")
    dhidden = made(dhidden, "dhidden", hidden is not None, r.shape, dy.dtype, "as many elements as r")
    dweight = made(dweight, "dweight", weight is not None, (H,), _F32, "H elements")
    dgate = made(dgate, "dgate", gate is not None, () if gate is None else gate.shape, _F32, "as many elements as gate")
    dpost_weight = made(dpost_weight, "dpost_weight", post_weight is not None, (H,), _F32, "H elements")
    _ws, ws_ptr, ws_bytes = _scratch("fp8_residual_norm_backward_workspace", (rows, H, gates), r, workspace)
    _lib.call("fp8_residual_norm_backward", dy.data_ptr(), r.data_ptr(), 1 if rt is _F32 else 0, _ptr(hidden), h_elem,
              _ptr(gate), g_elem, gates, _ptr(post_weight), _ptr(weight), w_elem if weight is not None else p_elem,
              rstd.data_ptr(), _ptr(post_rstd) if post_weight is not None else None, _ptr(dr), dx.data_ptr(),
              _ptr(dhidden), _ptr(dgate), _ptr(dpost_weight), _ptr(dweight), rows, H, alpha, ws_ptr, ws_bytes,
              _stream(r))
    return dx, dhidden, dweight, dgate, dpost_weight


def fp8_linear_into(qx, qw, sx, sw, out, col0=0, out_kind=OUT_BF16, sy=None,
                    accum=ACC_EXACT):
    """fp8_linear writing into columns [col0, col0 + N) of an existing
    row-major output ``out`` [..., L] (L >= col0 + N): the row stride of the
    written block is L.  Nothing outside that column block is touched."""
    _need(qx, "qx", torch.uint8)
    dev = qx.device
    _need(qw, "qw", torch.uint8, dev)
    K = qx.shape[-1]
    N = qw.shape[0]
    if qw.dim() != 2 or qw.shape[1] != K:
        raise ValueError("qw must be [N, K] with qx [..., K]")
    M = math.prod(qx.shape[:-1])
    _scale(sx, "sx", dev)
    _scale(sw, "sw", dev)
    dtype = {OUT_BF16: torch.bfloat16, OUT_FP8: torch.uint8, OUT_F32: torch.float32}[out_kind]
    _need(out, "out", dtype, dev)
    L = out.shape[-1]
    if out.numel() != M * L or col0 < 0 or col0 + N > L:
        raise ValueError("out must be [..., L] with M rows and col0 + N <= L")
    if out_kind == OUT_FP8:
        _scale(sy, "sy", dev)
    base = out.data_ptr() + col0 * out.element_size()
    _lib.call("fp8_linear_ldc", _ptr(qx), _ptr(qw), ctypes.c_void_p(base), M, N, K, L,
              _ptr(sx), _ptr(sw), out_kind, _ptr(sy) if sy is not None else None,
              accum, _stream(qx))
    return out


def fp8_requantize_onto_max(qw, s_member, s_group, out=None):
    """Codes of qw re-quantized onto the largest scale of its group (the fused
    single-scale failure mode; comparison workloads only)."""
    _need(qw, "qw", torch.uint8)
    dev = qw.device
    _scale(s_member, "s_member", dev)
    _need(s_group, "s_group", torch.float32, dev)
    if out is None:
        out = torch.empty_like(qw)
    _need(out, "out", torch.uint8, dev)
    if out.numel() != qw.numel():
        raise ValueError("out must match qw")
    _lib.call("fp8_requantize_onto_max", _ptr(qw), _ptr(out), qw.numel(), _ptr(s_member),
              _ptr(s_group), s_group.numel(), _stream(qw))
    return out


def silu_mul_2in_fp8(g, u, s_out, out=None, alpha=None, beta=None):
    """E4M3 codes of g * sigmoid(alpha g) * (u + beta) at ``s_out``; g and u
    BF16 of equal shape.  Without alpha and beta this is plain SwiGLU
    (silu(g) * u); alpha is a gain inside the sigmoid, beta an offset on up."""
    _need(g, "g", torch.bfloat16)
    _need(u, "u", torch.bfloat16, g.device)
    if g.shape != u.shape:
        raise ValueError("g and u must have the same shape")
    _scale(s_out, "s_out", g.device)
    if out is None:
        out = torch.empty(g.shape, dtype=torch.uint8, device=g.device)
    _need(out, "out", torch.uint8, g.device)
    if out.numel() != g.numel():
        raise ValueError("out must have as many elements as g")
    if alpha is None and beta is None:
        _lib.call("silu_mul_2in_fp8", _ptr(g), _ptr(u), _ptr(out), g.numel(),
                  _ptr(s_out), _stream(g))
    else:
        _lib.call("silu_mul_2in_fp8_ab", _ptr(g), _ptr(u), _ptr(out), g.numel(),
                  _ptr(s_out), 1.0 if alpha is None else float(alpha),
                  0.0 if beta is None else float(beta), _stream(g))
    return out


def silu_mul_fp8(x, s_out, out=None, alpha=None, beta=None):
    """One-input SwiGLU-FP8: x BF16 [..., 2I] whose rows hold the I gate values
    followed by the I up values; returns E4M3 codes [..., I] of
    g * sigmoid(alpha g) * (u + beta) at ``s_out`` (alpha 1, beta 0 when
    omitted), bit for bit what silu_mul_2in_fp8 gives on the two halves."""
    _need(x, "x", torch.bfloat16)
    if x.dim() == 0 or x.shape[-1] % 2:
        raise ValueError("x must end in an even dimension [..., 2I]")
    _scale(s_out, "s_out", x.device)
    inter = x.shape[-1] // 2
    rows = math.prod(x.shape[:-1])
    if out is None:
        out = torch.empty((*x.shape[:-1], inter), dtype=torch.uint8, device=x.device)
    _need(out, "out", torch.uint8, x.device)
    if out.numel() != rows * inter:
        raise ValueError("out must hold [..., I] elements")
    _lib.call("silu_mul_fp8", _ptr(x), _ptr(out), rows, inter, _ptr(s_out),
              1.0 if alpha is None else float(alpha),
              0.0 if beta is None else float(beta), _stream(x))
    return out


def fp8_gate_up_swiglu(qx, wg, sx, sg, wu, su, sh, out=None, accum=ACC_EXACT):
    """qh = SwiGLU-FP8 of the gate and up projections of an E4M3 activation
    qx [..., H] (wg, wu [I, H]); bitwise what fp8_linear (BF16 out) twice and
    silu_mul_2in_fp8 give when I >= H (with H > I and few tiles fp8_linear
    sums K in two halves and a code can differ by one step), in one kernel."""
    _need(qx, "qx", torch.uint8)
    dev = qx.device
    _need(wg, "wg", torch.uint8, dev)
    _need(wu, "wu", torch.uint8, dev)
    H = qx.shape[-1]
    I = wg.shape[0]
    if wg.shape != (I, H) or wu.shape != (I, H):
        raise ValueError("shapes: qx [..., H]; wg, wu [I, H]")
    for t, n in ((sx, "sx"), (sg, "sg"), (su, "su"), (sh, "sh")):
        _scale(t, n, dev)
    M = math.prod(qx.shape[:-1])
    if out is None:
        out = torch.empty((*qx.shape[:-1], I), dtype=torch.uint8, device=dev)
    _need(out, "out", torch.uint8, dev)
    if out.numel() != M * I:
        raise ValueError("out must hold M * I elements")
    _lib.call("fp8_gate_up_swiglu", _ptr(qx), _ptr(wg), _ptr(sx), _ptr(sg),
              _ptr(wu), _ptr(su), _ptr(sh), _ptr(out), M, I, H, accum, _stream(qx))
    return out


def gated_mlp_fp8_workspace(M, H, I):
    return int(_lib.lib().gated_mlp_fp8_workspace(M, H, I))


def _workspace(nbytes, device, ws):
    if ws is None:
        # 256-byte aligned: the caching allocator aligns blocks to 512 bytes
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    _need(ws, "workspace", torch.uint8, device)
    return ws


def gated_mlp_fp8(x, sx, wg, sg, wu, su, sh, wd, sd, out=None, workspace=None,
                  accum=ACC_EXACT):
    """Split gate/up gated MLP; x [..., H] BF16 -> y [..., H] BF16."""
    _need(x, "x", torch.bfloat16)
    dev = x.device
    for t, n in ((wg, "wg"), (wu, "wu"), (wd, "wd")):
        _need(t, n, torch.uint8, dev)
    H = x.shape[-1]
    I = wg.shape[0]
    if wg.shape != (I, H) or wu.shape != (I, H) or wd.shape != (H, I):
        raise ValueError("shapes: wg, wu [I, H]; wd [H, I]")
    for t, n in ((sx, "sx"), (sg, "sg"), (su, "su"), (sh, "sh"), (sd, "sd")):
        _scale(t, n, dev)
    M = math.prod(x.shape[:-1])
    if out is None:
        out = torch.empty(x.shape, dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, dev)
    if out.numel() != M * H:
        raise ValueError("out must hold M * H elements")
    nb = gated_mlp_fp8_workspace(M, H, I)
    ws = _workspace(nb, dev, workspace)
    _lib.call("gated_mlp_fp8", _ptr(x), M, H, I, _ptr(sx), _ptr(wg), _ptr(sg),
              _ptr(wu), _ptr(su), _ptr(sh), _ptr(wd), _ptr(sd), _ptr(out),
              _ptr(ws), ws.numel(), accum, _stream(x))
    return out


NOALLOC_SCRATCH_BYTES = 64 << 20   # FP8MOT_NOALLOC_SCRATCH_BYTES


def gated_mlp_fp8_noalloc(x, sx, wg, sg, wu, su, sh, wd, sd, out, accum=ACC_EXACT):
    """gated_mlp_fp8 without a workspace: the library keeps qX and qH in its
    own per-device scratch (at most NOALLOC_SCRATCH_BYTES); the caller passes
    the output.  Calls that overlap on one GPU race on that scratch."""
    _need(x, "x", torch.bfloat16)
    dev = x.device
    for t, n in ((wg, "wg"), (wu, "wu"), (wd, "wd")):
        _need(t, n, torch.uint8, dev)
    H = x.shape[-1]
    I = wg.shape[0]
    if wg.shape != (I, H) or wu.shape != (I, H) or wd.shape != (H, I):
        raise ValueError("shapes: wg, wu [I, H]; wd [H, I]")
    for t, n in ((sx, "sx"), (sg, "sg"), (su, "su"), (sh, "sh"), (sd, "sd")):
        _scale(t, n, dev)
    M = math.prod(x.shape[:-1])
    _need(out, "out", torch.bfloat16, dev)
    if out.numel() != M * H:
        raise ValueError("out must hold M * H elements")
    _lib.call("gated_mlp_fp8_noalloc", _ptr(x), M, H, I, _ptr(sx), _ptr(wg), _ptr(sg),
              _ptr(wu), _ptr(su), _ptr(sh), _ptr(wd), _ptr(sd), _ptr(out), accum,
              _stream(x))
    return out


def qkv_fp8_workspace(M, H):
    return int(_lib.lib().qkv_fp8_workspace(M, H))


def qkv_fp8(x, sx, wq, sq, wk, sk, wv, sv, outs=None, workspace=None,
            accum=ACC_EXACT):
    """Split Q/K/V over one shared quantization; returns (yq, yk, yv)."""
    _need(x, "x", torch.bfloat16)
    dev = x.device
    H = x.shape[-1]
    for t, n in ((wq, "wq"), (wk, "wk"), (wv, "wv")):
        _need(t, n, torch.uint8, dev)
        if t.dim() != 2 or t.shape[1] != H:
            raise ValueError(f"{n} must be [N, H]")
    for t, n in ((sx, "sx"), (sq, "sq"), (sk, "sk"), (sv, "sv")):
        _scale(t, n, dev)
    M = math.prod(x.shape[:-1])
    if outs is None:
        outs = tuple(torch.empty((*x.shape[:-1], w.shape[0]), dtype=torch.bfloat16,
                                 device=dev) for w in (wq, wk, wv))
    for o, w, n in zip(outs, (wq, wk, wv), ("yq", "yk", "yv")):
        _need(o, n, torch.bfloat16, dev)
        if o.numel() != M * w.shape[0]:
            raise ValueError(f"{n} must hold M * N elements")
    ws = _workspace(qkv_fp8_workspace(M, H), dev, workspace)
    yq, yk, yv = outs
    _lib.call("qkv_fp8", _ptr(x), M, H, _ptr(sx), _ptr(wq), wq.shape[0],
              _ptr(sq), _ptr(wk), wk.shape[0], _ptr(sk), _ptr(wv), wv.shape[0],
              _ptr(sv), _ptr(yq), _ptr(yk), _ptr(yv), _ptr(ws), ws.numel(),
              accum, _stream(x))
    return yq, yk, yv


def new_observer_state(device):
    """A fresh (zero-filled) 16-byte observer state on ``device``."""
    return torch.zeros(4, dtype=torch.int32, device=device)


def fp8_observe(x, state, mode=OBS_MAX, c=0.01):
    """Fold amax(|x|) of one calibration call into ``state``."""
    _need(x, "x", torch.bfloat16)
    _need(state, "state", torch.int32, x.device)
    if state.numel() != 4:
        raise ValueError("state must be a 16-byte observer state")
    _lib.call("fp8_observe", _ptr(x), x.numel(), _ptr(state), mode, c,
              _stream(x))
    return state


def fp8_observe_swiglu(g, u, state, mode=OBS_MAX, c=0.01):
    """Fold amax(|silu(g) * u|) into ``state``."""
    _need(g, "g", torch.bfloat16)
    _need(u, "u", torch.bfloat16, g.device)
    if g.shape != u.shape:
        raise ValueError("g and u must have the same shape")
    _need(state, "state", torch.int32, g.device)
    if state.numel() != 4:
        raise ValueError("state must be a 16-byte observer state")
    _lib.call("fp8_observe_swiglu", _ptr(g), _ptr(u), g.numel(), _ptr(state),
              mode, c, _stream(g))
    return state


def fp8_scale_from_state(state, out=None):
    """Static scale m / 448 from an observer state (one float32 on device)."""
    _need(state, "state", torch.int32)
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=state.device)
    _need(out, "out", torch.float32, state.device)
    _lib.call("fp8_scale_from_state", _ptr(state), _ptr(out), _stream(state))
    return out


def fp8_check_shared_scale(scales):
    """Load-time check: raises Fp8motError unless all scales are equal,
    finite and > 0.  ``scales`` is a host sequence of floats."""
    n = len(scales)
    arr = (ctypes.c_float * max(n, 1))(*[float(s) for s in scales])
    _lib.call("fp8_check_shared_scale", arr, n)


def rw_ceiling(a, b, out):
    """Measurement aid: the quantize (b None) or SwiGLU (b given) byte mix with
    no arithmetic; out[i] = low byte of a[i] (^ b[i]).  a, b: 16-bit tensors
    (any 2-byte dtype), out: uint8 with as many elements."""
    if a.element_size() != 2 or (b is not None and b.element_size() != 2):
        raise ValueError("a and b must hold 2-byte elements")
    for t, n in ((a, "a"), (out, "out")) + (((b, "b"),) if b is not None else ()):
        if t.device.type != "cuda" or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous GPU tensor")
    if out.dtype != torch.uint8 or out.numel() != a.numel() or (
            b is not None and b.numel() != a.numel()):
        raise ValueError("out must be uint8 with as many elements as a (and b)")
    _lib.call("fp8mot_rw_ceiling", _ptr(a), _ptr(b), _ptr(out), a.numel(), _stream(a))
    return out


def mfma_ceiling(a, b, iters, sink, accum=ACC_EXACT):
    """Measurement aid: 8 * iters dense MFMAs per wave on fragments built from
    the E4M3 codes in a and b (uint8 GPU tensors, indices wrapped), with
    nothing else in the loop; accum selects the F16 (exact engine) or the
    native FP8 instruction.  sink: one float32 GPU element, written only if
    the products sum to a sentinel.  Returns the launch's FLOP count."""
    _need(a, "a", torch.uint8)
    _need(b, "b", torch.uint8, a.device)
    _need(sink, "sink", torch.float32, a.device)
    flops = ctypes.c_double(0.0)
    _lib.call("fp8mot_mfma_ceiling", _ptr(a), a.numel(), _ptr(b), b.numel(), int(iters),
              int(accum), _ptr(sink), ctypes.byref(flops), _stream(a))
    return flops.value


def convert_f32(x, kind=CONV_E4M3_PACKED, out=None):
    """Verification aid: the kernels' FP32 -> E4M3 (kind CONV_E4M3_PACKED or
    CONV_E4M3_INT; uint8 codes) or FP32 -> BF16 (CONV_BF16; bfloat16 bits)
    conversion of every element of the float32 GPU tensor x (numel a
    multiple of 4).  Returns out (allocated when None)."""
    _need(x, "x", torch.float32)
    dtype = torch.bfloat16 if kind == CONV_BF16 else torch.uint8
    if out is None:
        out = torch.empty(x.shape, dtype=dtype, device=x.device)
    else:
        _need(out, "out", dtype, x.device)
        if out.numel() != x.numel():
            raise ValueError("out must have as many elements as x")
    _lib.call("fp8mot_convert_f32", _ptr(x), _ptr(out), x.numel(), int(kind), _stream(x))
    return out


def debug_quant_launches():
    return int(_lib.lib().fp8mot_debug_quant_launches())


def init(device=0):
    _lib.call("fp8mot_init", int(device))


def rtn_weight(w, state=None):
    """RTN per-tensor E4M3 weight with scale amax/448, on the GPU:
    fp8_observe (max) -> fp8_scale_from_state -> fp8_quant_static."""
    st = new_observer_state(w.device)
    fp8_observe(w, st, OBS_MAX)
    s = fp8_scale_from_state(st)
    return fp8_quant_static(w, s), s
