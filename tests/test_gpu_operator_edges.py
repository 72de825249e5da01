"""Calls of the operators around the sketch layer that have nothing to do, or
little: empty batches, odd but allowed shapes, and the forms that other tests
do not reach."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [False, True])
def test_an_empty_batch_has_no_flags(given):
    """No users: the flags are those of this call, not what the memory held."""
    import torch
    from sketch_attention_compression_b200 import (linear_attention_backward, linear_attention_forward,
                                                   read_device_status)
    q = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    g, off = torch.tensor([-0.1, -0.2]).cuda(), torch.zeros(1, dtype=torch.int64, device="cuda")
    for backward in (False, True):
        held = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
                for n in (256, 4096, 8192, 1 << 20) for _ in range(4)]
        ws = held.pop() if given else None
        del held
        if backward:
            grads, ws = linear_attention_backward(q, q, q, g, off, 0.1, q, workspace=ws)
            assert all(t.shape == q.shape for t in grads.values())
        else:
            out, state, ws = linear_attention_forward(q, q, q, g, off, 0.1, workspace=ws)
            assert out.shape == q.shape and state.shape == (0, 2, 64, 64)
        assert read_device_status(ws) == 0
