"""moe_orthogonalize checks `steps` before it becomes a C int (host only)."""
import pytest
import torch

import sparse_mixture_experts_16_b200 as moe


@pytest.mark.parametrize("steps", [2 ** 32 + 5, 5 - 2 ** 32, 0, -1, 17, 2.5])
@pytest.mark.parametrize("shape", [(2, 4, 4), (0, 4, 4)], ids=str)
def test_steps_that_are_not_1_to_16_are_refused(shape, steps):
    """2^32 + 5 and 5 - 2^32 have the lower 32 bits of 5"""
    with pytest.raises(moe.MoeError, match="INVALID_ARG"):
        moe.moe_orthogonalize(torch.zeros(shape), steps=steps)
