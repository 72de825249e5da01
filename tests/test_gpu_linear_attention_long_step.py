"""A stored state that is advanced row by row over a whole horizon."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("slots", [False, True])
def test_thousands_of_steps_do_not_drift(slots):
    """6000 rows at horizons of 1000 to 4096 rows, against the recurrence in 64
    bits.  Of each row's own roundings (three of at most 2^-24, in random
    directions) the last 4096 count, so the state is off by some sqrt(4096)
    2^-24, with a margin of two 2^-17; a decay that is off by 2^-25 in one
    direction would be off by 4096 times that, 2^-13."""
    import torch
    from sketch_attention_compression_b200 import linear_attention_step
    decay = torch.tensor([-0.00031, -0.00025, -0.00071, -0.00099])
    gen = torch.Generator().manual_seed(2)
    rows, heads, dk, dv = 6000, 4, 8, 16
    q, k = (torch.randn((rows, heads, dk), generator=gen) for _ in range(2))
    v = torch.randn((rows, heads, dv), generator=gen)
    state = torch.zeros((2, heads, dk, dv), device="cuda")
    where = torch.ones(1, dtype=torch.int64, device="cuda") if slots else None
    g, dq, dk_, dv_ = (t.cuda() for t in (decay, q, k, v))
    S = np.zeros((heads, dk, dv))
    l = np.exp(decay.double().numpy())[:, None, None]
    for t in range(rows):
        out = linear_attention_step(state, dq[t:t + 1], dk_[t:t + 1], dv_[t:t + 1], g, 0.25, slots=where)
        S = l * S + k[t].double().numpy()[:, :, None] * v[t].double().numpy()[:, None, :]
    got = state[int(slots)].double().cpu().numpy()
    for h in range(heads):
        err = np.linalg.norm(got[h] - S[h]) / np.linalg.norm(S[h])
        assert err < 2.0 ** -17, (h, err)
    want = 0.25 * np.einsum("hd,hde->he", q[-1].double().numpy(), S)
    assert np.linalg.norm(out[0].double().cpu().numpy() - want) <= 2.0 ** -16 * np.linalg.norm(want)


def test_an_infinite_state_stays_infinite():
    """Decays whose fp32 value is exact, rounded up and rounded down."""
    import torch
    from sketch_attention_compression_b200 import linear_attention_step
    g = torch.tensor([0.0, -0.00031, -0.00025, -0.3]).cuda()
    state = torch.full((1, 4, 4, 4), float("inf"), device="cuda")
    state[:, :, 1] = -float("inf")
    state[:, :, 2] = 3e38
    one = torch.ones((1, 4, 4), device="cuda")
    linear_attention_step(state, one, one, one, g, 1.0)
    assert (state[:, :, 0] == float("inf")).all() and (state[:, :, 1] == -float("inf")).all()
    assert torch.isfinite(state[:, :, 2]).all()


def test_a_state_without_decay_adds_one_rounding():
    """S + k v is one product and one sum: ties go to the even neighbour in
    either direction, and k = 0 leaves every bit."""
    import torch
    from sketch_attention_compression_b200 import linear_attention_step
    big = 2.0 ** 23
    state = torch.tensor([big, big + 1, -big, -big - 1, 1e-38, -3e38, 0.0, 1.0]).cuda()
    state = state.view(1, 1, 8, 1).expand(1, 1, 8, 4).contiguous()
    before = state.clone()
    k = torch.tensor([0.5, 0.5, 0.5, 0.5, 0.0, 0.0, 0.25, 0.0]).cuda().view(1, 1, 8)
    one, zero = torch.ones((1, 1, 4), device="cuda"), torch.zeros(1, device="cuda")
    linear_attention_step(state, k, k, one, zero, 1.0)
    want = before.double() + k.double().view(1, 1, 8, 1)
    assert torch.equal(state, want.float())  # (rounds once, to nearest even)
    again = state.clone()
    linear_attention_step(again, k, torch.zeros_like(k), one, zero, 1.0)
    assert torch.equal(again, state)
