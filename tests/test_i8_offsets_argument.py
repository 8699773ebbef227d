"""quantize_i8 takes its row count from the last offset: offsets without one are refused, as an empty
tensor's null address would mean all rows (no GPU needed)."""
import pytest
import torch

import block_scaled_fp4_04_b200 as fp4


@pytest.mark.parametrize("n", [0, 1])
def test_offsets_of_no_expert_are_refused(n):
    with pytest.raises(ValueError, match="offsets must be"):
        fp4.quantize_i8(torch.zeros(4, 64), torch.zeros(n, dtype=torch.int32))


def test_offsets_of_one_expert_are_taken():
    with pytest.raises(ValueError, match="CUDA tensors"):  # refused for where it is, not for its offsets
        fp4.quantize_i8(torch.zeros(4, 64), torch.zeros(2, dtype=torch.int32))
