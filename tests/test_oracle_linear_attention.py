"""Pins for the linear attention and block norm oracles: closed forms and
central differences (64 bits: truncation h^2 and rounding eps / h of the
difference are both below 1e-8 of the values at h = 1e-5)."""

import numpy as np
import pytest

from oracle import (block_norm, block_norm_grad, linear_attention, linear_attention_grad,
                    linear_attention_step)

OFFSETS = np.array([0, 4, 4, 9])
H, DK, DV = 2, 3, 2


def _inputs(seed):
    rng = np.random.default_rng(seed)
    n, b = int(OFFSETS[-1]), len(OFFSETS) - 1
    return (rng.standard_normal((n, H, DK)), rng.standard_normal((n, H, DK)),
            rng.standard_normal((n, H, DV)), np.array([-0.3, 0.0]),
            rng.standard_normal((b, H, DK, DV)), rng.standard_normal((n, H, DV)),
            rng.standard_normal((b, H, DK, DV)))


def _difference(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        y = x.copy()
        y[i] += h
        up = f(y)
        y[i] -= 2 * h
        g[i] = (up - f(y)) / (2 * h)
    return g


def test_closed_form():
    q, k, v, g, S0, _, _ = _inputs(1)
    out, fin = linear_attention(q, k, v, g, OFFSETS, 0.5, S0)
    for b in range(3):
        lo, hi = OFFSETS[b], OFFSETS[b + 1]
        for h in range(H):
            for t in range(lo, hi):
                want = 0.5 * np.exp(g[h] * (t - lo + 1)) * q[t, h] @ S0[b, h]
                for j in range(lo, t + 1):
                    want = want + 0.5 * np.exp(g[h] * (t - j)) * (q[t, h] @ k[j, h]) * v[j, h]
                np.testing.assert_allclose(out[t, h], want, rtol=1e-12, atol=1e-13)
    np.testing.assert_array_equal(fin[1], S0[1])


def test_steps_equal_the_scan():
    q, k, v, g, S0, _, _ = _inputs(2)
    out, fin = linear_attention(q, k, v, g, [0, 9], 0.7, S0[:1])
    S = S0[:1]
    for t in range(9):
        o, S = linear_attention_step(S, q[t:t + 1], k[t:t + 1], v[t:t + 1], g, 0.7)
        np.testing.assert_array_equal(o[0], out[t])
    np.testing.assert_array_equal(S, fin)


@pytest.mark.parametrize("which", range(4))
def test_attention_gradients_against_differences(which):
    q, k, v, g, S0, do, dS = _inputs(3)
    args = [q, k, v, S0]

    def loss(x):
        a = list(args)
        a[which] = x
        out, fin = linear_attention(a[0], a[1], a[2], g, OFFSETS, 0.5, a[3])
        return (out * do).sum() + (fin * dS).sum()

    got = linear_attention_grad(q, k, v, g, OFFSETS, 0.5, do, S0, dS)
    name = ("dq", "dk", "dv", "d_initial_state")[which]
    np.testing.assert_allclose(got[name], _difference(loss, args[which]), rtol=1e-7, atol=1e-7)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("gate_kind", ["identity", "sigmoid", "silu"])
def test_norm_gradients_against_differences(kind, gate_kind):
    rng = np.random.default_rng(5)
    n, d = 3, 5
    p = {key: rng.standard_normal((n, d)) for key in ("x", "y", "z")}
    p |= {key: rng.standard_normal(d) for key in ("g1", "b1", "rs", "g2", "b2")}
    dr, du = rng.standard_normal((n, d)), rng.standard_normal((n, d))

    def loss(name, value):
        r, u = block_norm(**{**p, name: value}, kind=kind, gate_kind=gate_kind)
        return (r * dr).sum() + (u * du).sum()

    r, _ = block_norm(**p, kind=kind, gate_kind=gate_kind)
    rest = {key: p[key] for key in ("z", "g1", "b1", "rs", "g2", "b2")}
    got = block_norm_grad(r, p["y"], dr, du, **rest, kind=kind, gate_kind=gate_kind)
    names = dict(x="d_residual", y="d_block", z="d_gate", g1="d_post_gain", b1="d_post_bias",
                 rs="d_res_scale", g2="d_pre_gain", b2="d_pre_bias")
    assert set(names.values()) == set(got)
    for key, name in names.items():
        want = _difference(lambda v, key=key: loss(key, v), p[key])
        np.testing.assert_allclose(got[name], want, rtol=1e-6, atol=1e-7)


def test_norm_closed_values():
    x = np.array([[3.0, 1.0]])
    assert block_norm(x, g2=np.ones(2), eps=0.0)[1].tolist() == [[1.0, -1.0]]
    u = block_norm(x, g2=np.ones(2), kind="rms", eps=0.0)[1]
    np.testing.assert_allclose(u, x / np.sqrt(5.0))
    assert block_norm(x)[0] is None
