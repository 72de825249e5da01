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


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("batch", [1024, 5461, 5462, 7003])
def test_many_entries_with_slots(batch, dtype):
    """Batches around the size (16384 blocks) from which equal slots are looked for ahead of
    the step: pairs that are neighbours, far apart and at both ends, slots
    taken three times, padded entries and slots past the pool."""
    import torch
    from oracle import linear_attention_step as oracle
    from sketch_attention_compression_b200 import linear_attention_step
    gen = torch.Generator().manual_seed(batch)
    t, states, heads, dk, dv = getattr(torch, dtype), batch + 5, 3, 4, 8
    q, k = (torch.randn((batch, heads, dk), generator=gen).to(t) for _ in range(2))
    v, s0 = torch.randn((batch, heads, dv), generator=gen).to(t), torch.randn((states, heads, dk, dv),
                                                                               generator=gen)
    slots = torch.randperm(states, generator=gen)[:batch]
    for later, earlier in ((batch - 1, 0), (1, 0), (33, 32), (64, 31), (700, 3), (701, 3), (900, 899)):
        slots[later] = slots[earlier]
    slots[5], slots[6], slots[500], slots[800] = -1, -7, states, 1 << 40
    g = torch.tensor([-0.1, 0.0, -3.0])
    state, flags = s0.clone().cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((batch, heads, dv), float("nan"), dtype=t, device="cuda")
    linear_attention_step(state, q.cuda(), k.cuda(), v.cuda(), g.cuda(), 0.5, slots=slots.cuda(), out=out,
                          device_flags=flags)
    taken, seen = [], set()
    for s in slots.tolist():
        ok = 0 <= s < states and s not in seen
        seen.add(s)
        taken.append(s if ok else -1)
    assert taken.count(-1) == 7 + 4 and flags.item() == 128
    want, after = oracle(s0.numpy(), *(x.double().numpy() for x in (q, k, v, g)), 0.5, taken)
    half = 2.0 ** -8 if dtype == "bfloat16" else 0.0
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= half * np.abs(want) + 16 * 2.0 ** -24 * 64).all()  # |terms| < 64 in all
    assert (out[[i for i, s in enumerate(taken) if s < 0]] == 0).all()
    assert np.abs(state.double().cpu().numpy() - after).max() <= 4 * 2.0 ** -24 * 16
    again = s0.clone().cuda()
    both = torch.empty_like(out)
    graph = torch.cuda.CUDAGraph()
    args = [x.cuda() for x in (q, k, v, g)], slots.cuda()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        linear_attention_step(again, *args[0], 0.5, slots=args[1], out=both)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(both, out) and torch.equal(again, state)


@pytest.mark.parametrize("batch", [40, 5600])
def test_a_step_whose_output_replaces_v(batch):
    """An entry's output may take its v's place, however equal slots are found."""
    import torch
    from sketch_attention_compression_b200 import linear_attention_step
    gen = torch.Generator().manual_seed(batch)
    q, k, v = (torch.randn((batch, 3, 8), generator=gen).cuda() for _ in range(3))
    s0, g = torch.randn((batch, 3, 8, 8), generator=gen).cuda(), torch.tensor([-0.1, 0.0, -2.0]).cuda()
    slots = torch.randperm(batch, generator=gen).cuda()
    slots[7] = slots[3]
    one, two = s0.clone(), s0.clone()
    want = linear_attention_step(one, q, k, v, g, 0.5, slots=slots)
    got = linear_attention_step(two, q, k, v, g, 0.5, slots=slots, out=v)
    assert got.data_ptr() == v.data_ptr() and torch.equal(got, want) and torch.equal(one, two)
