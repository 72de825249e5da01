"""The norms around a block with its gate and residual scale, in 64 bits:

    r = x + rs * act(z) * norm(y; g1, b1),   u = norm(r; g2, b2)
"""

from __future__ import annotations

import numpy as np


def _normalise(x, kind, eps):
    """(x^, rstd): the normalised rows and their inverse deviations."""
    if kind == "layer":
        x = x - x.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * rstd, rstd


def _act(z, kind):
    """(act(z), act'(z))."""
    if kind == "identity":
        return z, np.ones_like(z)
    s = 1.0 / (1.0 + np.exp(-z))
    return (s, s * (1 - s)) if kind == "sigmoid" else (z * s, s * (1 + z * (1 - s)))


def _norm_grad(x, kind, eps, d):
    """Gradient of the normalised rows at x for the upstream d."""
    hat, rstd = _normalise(x, kind, eps)
    mean = d.mean(-1, keepdims=True) if kind == "layer" else 0.0
    return rstd * (d - mean - hat * (d * hat).mean(-1, keepdims=True))


def block_norm(x, y=None, z=None, g1=None, b1=None, rs=None, g2=None, b2=None, kind="layer",
               gate_kind="identity", eps=1e-5):
    """(r, u); None for what is not computed."""
    r = x
    if y is not None:
        n = y if g1 is None else _normalise(y, kind, eps)[0] * g1 + (0 if b1 is None else b1)
        r = x + (1 if rs is None else rs) * (1 if z is None else _act(z, gate_kind)[0]) * n
    u = None if g2 is None else _normalise(r, kind, eps)[0] * g2 + (0 if b2 is None else b2)
    return (None if y is None else r), u


def block_norm_grad(r, y=None, dr=None, du=None, z=None, g1=None, b1=None, rs=None, g2=None,
                    b2=None, kind="layer", gate_kind="identity", eps=1e-5):
    """The gradients at the residual output r, by operand."""
    out, dx = {}, np.zeros_like(r) if dr is None else np.array(dr)
    if du is not None:
        hat = _normalise(r, kind, eps)[0]
        out["d_pre_gain"] = (du * hat).sum(0)
        if b2 is not None:
            out["d_pre_bias"] = du.sum(0)
        dx = dx + _norm_grad(r, kind, eps, du * g2)
    out["d_residual"] = dx
    if y is None:
        return out
    hat = y if g1 is None else _normalise(y, kind, eps)[0]
    n = y if g1 is None else hat * g1 + (0 if b1 is None else b1)
    act, slope = (1.0, 0.0) if z is None else _act(z, gate_kind)
    scale = 1.0 if rs is None else rs
    if z is not None:
        out["d_gate"] = dx * scale * n * slope
    if rs is not None:
        out["d_res_scale"] = (dx * act * n).sum(0)
    dn = dx * scale * act
    if g1 is not None:
        out["d_post_gain"] = (dn * hat).sum(0)
        if b1 is not None:
            out["d_post_bias"] = dn.sum(0)
        dn = _norm_grad(y, kind, eps, dn * g1)
    out["d_block"] = dn
    return out
