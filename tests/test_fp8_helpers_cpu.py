"""What the helpers around the calls on 8-bit floating-point blocks refuse before any call."""

import pytest
import torch

from expert_serving_amd import abi


@pytest.mark.parametrize("shape", [(256,), (2, 3, 128, 256), (1, 1, 1, 128, 128)])
def test_weights_are_matrices(shape):
    """A tensor of other dimensions than [N, K] and [E, N, K] is refused rather than quantised in part."""
    with pytest.raises(ValueError, match="N, K"):
        abi.quantize_fp8_weights(torch.ones(shape))
