"""CPU: block codes are refused over x, also where both take as many bytes.  No
kernel runs, no pointer is dereferenced."""

import ctypes

import pytest

from mlp_fp8_quant_amd import _lib as L

P = ctypes.c_void_p
NULL, INVALID = P(0), 1
X, W, SCALES = P(1 << 20), P(2 << 20), P(3 << 20)


@pytest.mark.parametrize("elem,H", [(0, 8), (1, 4), (0, 7), (0, 16), (1, 3)])
def test_block_codes_over_x(elem, H):
    # rows of 8 BF16 or 4 FP32 are 16 bytes, as many as their padded codes
    f = L.lib().fp8_residual_norm
    assert f(X, elem, NULL, 0, NULL, 0, 1, NULL, W, 0, NULL, X, 3, NULL, SCALES, NULL, NULL, 4, H, 1.0, 1e-6,
             NULL) == INVALID
