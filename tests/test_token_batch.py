"""A number of sequences past the C ABI's 32-bit field, which the binding of the token operators refuses. No GPU needed."""
import pytest
import torch

from submanifold_sparse_conv_amd import tokens


@pytest.mark.parametrize("batch", [1 << 31, (1 << 32) + 1])
def test_sequences_past_their_field(batch):
    cu = torch.empty(batch + 1, dtype=torch.int32)  # never touched
    with pytest.raises(ValueError, match="sequences"):
        tokens._window(cu, cu, None, -1, 0, 0, None, 64, cu.device)
