"""CPU: a workspace that lies over another tensor of its call is refused, as an
output that does so is.  No kernel runs, no pointer is dereferenced."""

import ctypes

import pytest

from mlp_fp8_quant_amd import _lib as L

P = ctypes.c_void_p
NULL, INVALID = P(0), 1


def at(i, byte=0):
    return P((i << 32) + byte)             # a tensor of its own, 4 GiB apart


def call(f, tensors, over, ws_bytes, build):
    """f's status with its workspace at the start, inside and just before the
    end of each tensor named in ``over`` (name -> bytes)."""
    for name, size in over.items():
        for shift in {0, size // 32 * 16, max(0, size - 16) // 16 * 16}:
            ws = P(tensors[name].value + shift)
            assert f(*build(tensors, ws)) == INVALID, (name, shift)
        # a workspace whose last bytes reach into the tensor
        ws = P(tensors[name].value - (ws_bytes - 16) // 16 * 16)
        assert f(*build(tensors, ws)) == INVALID, name


@pytest.mark.parametrize("rows", [0, 1])
def test_linear(rows):
    lib = L.lib()
    M, N, K = 3000, 700, 4000
    need = lib.fp8_linear_act_workspace(M, N, K)
    assert need == 3 * M * N * 4
    names = ["qx", "qw", "y", "sx", "sw", "bias", "res", "pre", "sy"]
    t = {n: at(i + 1) for i, n in enumerate(names)}
    over = dict(qx=M * K, qw=N * K, y=M * N, sx=4 * M if rows else 4, sw=4 * N if rows else 4, bias=4 * N, res=4 * M * N,
                pre=2 * M * N, sy=4)
    call(lib.fp8_linear_act, t, over, need, lambda t, ws: (
        t["qx"], t["qw"], t["y"], M, N, K, t["sx"], t["sw"], rows, t["bias"], 1, 1, t["res"], 1, t["pre"], 1, t["sy"], 0,
        ws, need, NULL))


def test_linear_backward():
    lib = L.lib()
    M, N = 4000, 520
    need = lib.fp8_linear_act_backward_workspace(M, N)
    assert need > 0
    t = {n: at(i + 1) for i, n in enumerate(["dy", "pre", "dz", "db"])}
    call(lib.fp8_linear_act_backward, t, dict(dy=2 * M * N, pre=2 * M * N, dz=2 * M * N, db=4 * N), need,
         lambda t, ws: (t["dy"], t["pre"], 4, t["dz"], t["db"], M, N, ws, need, NULL))


@pytest.mark.parametrize("rows,H", [(4000, 520), (7, 20000)])
def test_norm_backward(rows, H):
    lib = L.lib()
    need = lib.fp8_layer_norm_backward_workspace(rows, H)
    assert need > 0
    t = {n: at(i + 1) for i, n in enumerate(["dy", "x", "w", "mean", "rstd", "dres", "dx", "dw", "db"])}
    n = rows * H
    over = dict(dy=2 * n, x=4 * n, w=4 * H, mean=4 * rows, rstd=4 * rows, dres=4 * n, dx=4 * n, dw=4 * H, db=4 * H)
    call(lib.fp8_layer_norm_backward, t, over, need, lambda t, ws: (
        t["dy"], 0, t["x"], 1, t["w"], 1, t["mean"], t["rstd"], t["dres"], t["dx"], t["dw"], t["db"], rows, H, ws, need,
        NULL))
