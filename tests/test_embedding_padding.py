"""A padding index outside the vocabulary is refused where the lookup is called, not first in the backward pass."""
import pytest
import torch

from lora_fine_tuning_mlp_b200 import api


@pytest.mark.parametrize("padding", [-1, 10, 2 ** 40])
def test_refused_in_the_forward(padding):
    E = torch.zeros(10, 16, dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(ValueError, match="padding_idx"):
        api.EmbeddingFunction.apply(torch.zeros(4, dtype=torch.int64), E, 1.0, padding)
