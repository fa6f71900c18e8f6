"""A position past 32 bits is refused by the binding: as a C int it would be another position (no GPU: nothing is launched)."""

import pytest
import torch

from gated_linear_recurrence_conv1d_b200 import binding


@pytest.mark.parametrize("pos0", [2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1, 2 ** 40])
def test_positions_past_32_bits(pos0):
    d = binding.make_mqa_dims(2, 16, 3, 256, 8)
    x = torch.zeros(1)
    with pytest.raises(ValueError, match="pos0"):
        binding.mqa_forward(d, x, x, x, x, x, x, pos0=pos0)
    with pytest.raises(ValueError, match="pos0"):
        binding.mqa_cache8_write(d, x, x, x, x, pos0=pos0)
