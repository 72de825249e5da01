"""The gates' values and slopes over a wide range, relative to themselves.

The exponential of a rounded multiple of z is off by |z| 2^-24, the
approximate exponential and reciprocal by 2^-22 each, and a result passes
some eight further roundings: (|z| + 16) 2^-24 of the sum of the magnitudes
of its terms, and 2^-8 of itself more as bf16."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

E32, E16 = 2.0 ** -24, 2.0 ** -8


def _sigmoid(z):
    """sigmoid(z) and 1 - sigmoid(z), each to full relative precision."""
    t = np.exp(-np.abs(z))
    return np.where(z < 0, t, 1.0) / (1 + t), np.where(z < 0, 1.0, t) / (1 + t)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("kind", ["sigmoid", "silu"])
@pytest.mark.parametrize("d", [128, 100])
def test_gate_and_slope_over_their_range(kind, dtype, d):
    import torch
    from sketch_attention_compression_b200 import block_norm_backward, block_norm_forward
    t, rows = getattr(torch, dtype), 61
    z = torch.linspace(-30.0, 30.0, rows * d).view(rows, d).to(t).cuda()
    x = torch.zeros((rows, d), device="cuda")
    y, dr = torch.full_like(z, 2.0), torch.full_like(x, 0.5)
    r, _ = block_norm_forward(x, y, z, gate_kind=kind)
    got = block_norm_backward(r, y, dr, None, z, gate_kind=kind)
    zz = z.double().cpu().numpy()
    s, rest = _sigmoid(zz)
    act = s if kind == "sigmoid" else zz * s
    slope = s * rest if kind == "sigmoid" else s + zz * s * rest
    mag = s * rest if kind == "sigmoid" else s + np.abs(zz) * s * rest
    tol = (np.abs(zz) + 16) * E32
    half = E16 if dtype == "bfloat16" else 0.0
    err = np.abs(r.double().cpu().numpy() - 2 * act)
    assert (err <= tol * 2 * np.abs(act)).all()
    err = np.abs(got["d_gate"].double().cpu().numpy() - slope)  # 0.5 * 2 * slope
    assert (err <= tol * mag + half * np.abs(slope)).all(), (err / np.abs(slope)).max()
    err = np.abs(got["d_block"].double().cpu().numpy() - 0.5 * act)
    assert (err <= (tol + half) * 0.5 * np.abs(act)).all()


def test_gates_of_infinities_and_nan():
    import torch
    from sketch_attention_compression_b200 import block_norm_backward, block_norm_forward
    z = torch.zeros((2, 64), device="cuda")
    z[0, :3] = torch.tensor([float("inf"), -float("inf"), float("nan")])
    one = torch.ones_like(z)
    r, _ = block_norm_forward(torch.zeros_like(z), one, z, gate_kind="sigmoid")
    got = block_norm_backward(r, one, one, None, z, gate_kind="sigmoid")
    assert r[0, 0] == 1 and r[0, 1] == 0 and torch.isnan(r[0, 2]) and (r[0, 3:] == 0.5).all()
    assert (got["d_gate"][0, :2] == 0).all() and torch.isnan(got["d_gate"][0, 2])
    assert (got["d_gate"][0, 3:] == 0.25).all() and (got["d_gate"][1] == 0.25).all()
