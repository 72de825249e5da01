"""What the Python calls of the operators refuse before they look at a device
(CPU tensors; this runs without a GPU)."""

import pytest
import torch

from sketch_attention_compression_b200 import linear_attention_step


def _step(**change):
    q = torch.zeros((1, 2, 8))
    a = dict(state=torch.zeros((1, 2, 8, 8)), q=q, k=q, v=q, log_decay=torch.zeros(2), scale=1.0)
    return linear_attention_step(**{**a, **change})


@pytest.mark.parametrize("flags", [torch.zeros(0, dtype=torch.int32), torch.zeros(3, dtype=torch.uint8),
                                   torch.zeros(1, dtype=torch.int16)])
def test_flags_that_do_not_hold_a_word(flags):
    """The kernel's atomic writes four bytes."""
    with pytest.raises(ValueError, match="device_flags"):
        _step(device_flags=flags)
    with pytest.raises(ValueError, match="device"):  # a word, but no GPU tensors
        _step(device_flags=torch.zeros(1, dtype=torch.int32))
