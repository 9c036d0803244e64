"""CPU: the residual norms refuse numbers of gates that their sizes cannot count,
also for batches of no rows, which any number divides.  No kernel runs, no pointer
is dereferenced."""

import ctypes

import pytest

from mlp_fp8_quant_amd import _lib as L

P = ctypes.c_void_p
NULL, OK, INVALID = P(0), 0, 1


def at(i):
    return P(i << 40)


@pytest.mark.parametrize("gates", [0, -1, 1 << 31, 1 << 40, (1 << 62) + 1])
@pytest.mark.parametrize("rows", [0, 4])
def test_numbers_of_gates(rows, gates):
    lib = L.lib()
    assert lib.fp8_residual_norm(at(1), 0, at(2), 0, at(3), 0, gates, NULL, NULL, 0, at(4), at(5), 0, NULL, NULL, NULL,
                                 NULL, rows, 8, 1.0, 1e-6, NULL) == INVALID
    assert lib.fp8_residual_norm_backward_workspace(rows, 8, gates) == 0
    assert lib.fp8_residual_norm_backward(at(1), at(2), 0, at(3), 0, at(4), 0, gates, NULL, at(6), 0, at(7), NULL, NULL,
                                          at(8), at(9), at(10), NULL, at(11), rows, 8, 1.0, at(12), 1 << 30,
                                          NULL) == INVALID


def test_no_rows_of_many_gates():
    # nothing is asked for: nothing to do
    f = L.lib().fp8_residual_norm_backward
    assert f(NULL, NULL, 0, NULL, 0, at(4), 0, 1 << 20, NULL, at(6), 0, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, 0,
             8, 1.0, NULL, 0, NULL) == OK
