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


def test_a_step_of_one_key_column_in_any_layout():
    """d_k = 1: the stride of a dimension of one element is no stride."""
    import torch
    from sketch_attention_compression_b200 import linear_attention_step
    gen = torch.Generator().manual_seed(6)
    q, k = (torch.randn((1, 3, 2), generator=gen).cuda().permute(2, 1, 0) for _ in range(2))
    assert q.shape == (2, 3, 1) and q.stride(2) != 1
    v, s0 = torch.randn((2, 3, 8), generator=gen).cuda(), torch.randn((2, 3, 1, 8), generator=gen).cuda()
    g = torch.tensor([-0.1, 0.0, -2.0]).cuda()
    one, two = s0.clone(), s0.clone()
    a = linear_attention_step(one, q, k, v, g, 0.5)
    b = linear_attention_step(two, q.contiguous(), k.contiguous(), v, g, 0.5)
    assert torch.equal(a, b) and torch.equal(one, two)
    want = torch.exp(g.double())[:, None, None] * s0.double() + k.double()[..., None] * v.double()[:, :, None]
    assert np.abs((one.double() - want).cpu().numpy()).max() <= 4 * 2.0 ** -24 * want.abs().max().item()
