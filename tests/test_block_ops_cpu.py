"""CPU: the custom op of the residual norm refuses the output kind whose result it
cannot return, before any kernel runs."""

import pytest
import torch

import mlp_fp8_quant_amd as fp8
import mlp_fp8_quant_amd.torch_ops  # noqa: F401


@pytest.mark.parametrize("kind", [fp8.OUT_FP8_BLOCK, 7, -1])
def test_block_codes_have_an_op_of_their_own(kind):
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="out_kind"):
        torch.ops.fp8mot.residual_norm(x, x, None, None, None, 1.0, 1e-6, kind)
