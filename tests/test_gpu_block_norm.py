"""The norms around a block (forward and backward) against 64 bits.

Arithmetic is fp32 and a row's sums are trees of at most 8 * 2 sequential and
9 tree additions, so a value passes fewer than 64 roundings of 2^-24 relative
to the magnitudes below (sums of the absolute values of its terms; the gate's
exponential counts for 8 of them at |z| < 6).  An output of bf16 is rounded
once more (2^-8 of itself).  A sum over rows adds one rounding per row of a
thread and per block.
"""

import numpy as np
import pytest

from oracle import block_norm, block_norm_grad

pytestmark = pytest.mark.gpu

E32, E16 = 2.0 ** -24, 2.0 ** -8
NAMES = dict(z="gate", g1="post_gain", b1="post_bias", rs="res_scale", g2="pre_gain", b2="pre_bias")


def _make(rows, d, dtype, res, seed, kind="layer", gate=True, post=True, scale=True, pre=True):
    import torch
    gen = torch.Generator().manual_seed(seed)
    t = {"bf16": torch.bfloat16, "fp32": torch.float32}

    def draw(*shape, dtype=torch.float32, mul=1.0, add=0.0):
        return (torch.randn(shape, generator=gen) * mul + add).to(dtype)

    x = dict(x=draw(rows, d, dtype=t[res], mul=2.0, add=0.5), y=draw(rows, d, dtype=t[dtype], add=0.1),
             dr=draw(rows, d, dtype=t[res]), du=draw(rows, d, dtype=t[dtype]))
    if gate:
        x["z"] = draw(rows, d, dtype=t[dtype])
    if post:
        x["g1"] = draw(d, mul=0.2, add=1.0)
        if kind == "layer":
            x["b1"] = draw(d, mul=0.1)
    if scale:
        x["rs"] = draw(d, mul=0.1, add=0.5)
    if pre:
        x["g2"] = draw(d, mul=0.2, add=1.0)
        if kind == "layer":
            x["b2"] = draw(d, mul=0.1)
    else:
        del x["du"]
    return {k: v.cuda() for k, v in x.items()}, {k: v.double().numpy() for k, v in x.items()}


def _params(x):
    return {NAMES[k]: x.get(k) for k in NAMES}


def _magnitude_of_norm(x, kind, eps=1e-5):
    """|x^| with the terms of x - mean added up, at least 1 / rstd-scaled."""
    c = x - x.mean(-1, keepdims=True) if kind == "layer" else x
    rstd = 1 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    return rstd * (np.abs(x) + np.abs(x).mean(-1, keepdims=True)), rstd


def _rounded(tol, mag, want, dtype):
    return tol * mag + (E16 * np.abs(want) * (1 + 1e-3) if "bfloat16" in str(dtype) else 0) + 1e-36


def _near(got, want, mag, tol, what):
    g = got.double().cpu().numpy()
    err = np.abs(g - want)
    bad = err > _rounded(tol, mag, want, got.dtype)
    assert np.all(np.isfinite(g)) and not bad.any(), \
        f"{what}: {np.argwhere(bad)[:3].tolist()}, {(err / (mag + 1e-36)).max() / E32:.3g} x 2^-24"


def _check(rows, d, dtype, res, kind, gate_kind, seed=0, strides=None, **opts):
    from sketch_attention_compression_b200 import block_norm_backward, block_norm_forward
    import torch
    x, w = _make(rows, d, dtype, res, seed + rows + d, kind=kind, gate=gate_kind is not None, **opts)
    if strides is not None:
        for key in ("x", "y", "z", "dr", "du"):
            if key in x:
                wide = torch.full((rows, d + strides), float("nan"), dtype=x[key].dtype, device="cuda")
                wide[:, strides // 2:strides // 2 + d] = x[key]
                x[key] = wide[:, strides // 2:strides // 2 + d]
    kw = dict(kind=kind, gate_kind=gate_kind or "identity")
    p = _params(x)
    ow = {k: w.get(k) for k in NAMES}
    r, u = block_norm_forward(x["x"], x["y"], **p, **kw)
    wr, wu = block_norm(w["x"], w["y"], **ow, **kw)
    one = np.ones_like
    ab = {k: np.abs(v) for k, v in w.items()}
    my, _ = _magnitude_of_norm(w["y"], kind) if "g1" in w else (ab["y"], None)
    mn = my * ab.get("g1", one(my)) + ab.get("b1", 0)
    act = one(my) if "z" not in w else (ab["z"] if kw["gate_kind"] != "sigmoid" else one(my))
    mr = ab["x"] + ab.get("rs", 1) * act * mn
    _near(r, wr, mr, 64 * E32, "residual")
    if u is not None:
        # r's own error passes through the norm
        mu, rstd = _magnitude_of_norm(wr, kind)
        mu = (mu + rstd * (mr + mr.mean(-1, keepdims=True)) *
              (1 + mu)) * ab["g2"] + ab.get("b2", 0)
        _near(u, wu, mu, 64 * E32, "normed")
    else:
        assert wu is None
    # the gradients, at a residual that both sides hold exactly
    r64 = r.double().cpu().numpy()
    del p["pre_bias"]
    got = block_norm_backward(r, x["y"], x["dr"], x.get("du"), pre_bias=x.get("b2"), **p, **kw)
    want = block_norm_grad(r64, w["y"], w["dr"], w.get("du"), **ow, **kw)
    assert set(got) == set(want)
    mdx = ab["dr"].copy()
    if "du" in w:
        mh, rstd = _magnitude_of_norm(r64, kind)
        h = ab["du"] * ab["g2"]
        mdx = mdx + rstd * (h + h.mean(-1, keepdims=True) + 2 * mh * (h * mh).mean(-1, keepdims=True))
    slope = one(my) * 1.1
    mdn = mdx * ab.get("rs", 1) * act
    my1, ry = _magnitude_of_norm(w["y"], kind)
    p1 = mdn * ab.get("g1", 1)
    mag = dict(d_residual=mdx, d_gate=mdx * ab.get("rs", 1) * mn * slope * 2,
               d_block=mdn if "g1" not in w else
               ry * (p1 + p1.mean(-1, keepdims=True) + 2 * my1 * (p1 * my1).mean(-1, keepdims=True)),
               d_post_gain=(mdn * my).sum(0), d_post_bias=mdn.sum(0), d_res_scale=(mdx * act * mn).sum(0))
    if "du" in w:
        mag |= dict(d_pre_gain=(ab["du"] * mh).sum(0), d_pre_bias=ab["du"].sum(0))
    for name, val in got.items():
        _near(val, want[name], mag[name], (96 + rows / 4) * E32 if val.dim() == 1 else 96 * E32, name)


@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("d", [1, 7, 8, 31, 32, 64, 100, 128, 192, 256, 300, 1000, 1024, 2048, 4096,
                               4100, 8192])
def test_widths(d, dtype, res):
    _check(37, d, dtype, res, "layer", "silu")
    _check(5, d, dtype, res, "rms", "sigmoid", scale=False)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("gate_kind", [None, "identity", "sigmoid", "silu"])
@pytest.mark.parametrize("post,scale,pre", [(True, True, False), (False, True, True),
                                            (False, False, True), (True, False, True),
                                            (False, False, False)])
def test_every_combination(kind, gate_kind, post, scale, pre):
    _check(19, 96, "bf16", "fp32", kind, gate_kind, post=post, scale=scale, pre=pre)


@pytest.mark.parametrize("rows", [1, 2, 33, 5000])
@pytest.mark.parametrize("d,strides", [(128, None), (128, 8), (128, 3), (1024, 16), (40, 2)])
def test_rows_and_strides(rows, d, strides):
    _check(rows, d, "bf16", "bf16", "layer", "silu", strides=strides)


def test_only_the_next_blocks_norm():
    import torch
    from sketch_attention_compression_b200 import block_norm_backward, block_norm_forward
    x, w = _make(9, 64, "bf16", "fp32", 3)
    r, u = block_norm_forward(x["x"], pre_gain=x["g2"], pre_bias=x["b2"], dtype=torch.bfloat16)
    assert r is None and u.dtype == torch.bfloat16
    mu, _ = _magnitude_of_norm(w["x"], "layer")
    _near(u, block_norm(w["x"], g2=w["g2"], b2=w["b2"])[1], mu * np.abs(w["g2"]) + np.abs(w["b2"]),
          64 * E32, "normed")
    got = block_norm_backward(x["x"], None, None, x["du"], pre_gain=x["g2"], pre_bias=x["b2"])
    want = block_norm_grad(w["x"], None, None, w["du"], g2=w["g2"], b2=w["b2"])
    assert set(got) == set(want) == {"d_residual", "d_pre_gain", "d_pre_bias"}
    h = np.abs(w["du"] * w["g2"])
    _, rstd = _magnitude_of_norm(w["x"], "layer")
    mag = rstd * (h + h.mean(-1, keepdims=True) + 2 * mu * (h * mu).mean(-1, keepdims=True))
    _near(got["d_residual"], want["d_residual"], mag, 96 * E32, "d_residual")


def test_large_mean_constant_rows_and_not_finite_ones():
    """A large common offset loses nothing but the offset's own rounding; a
    constant row normalises to its bias; a row that is not finite stays alone."""
    import torch
    from sketch_attention_compression_b200 import block_norm_forward
    g = torch.Generator().manual_seed(1)
    x = (torch.randn((4, 256), generator=g) + 4096).cuda()
    one, b = torch.ones(256).cuda(), torch.full((256,), 0.25).cuda()
    want = block_norm(x.double().cpu().numpy(), g2=np.ones(256), b2=np.full(256, 0.25))[1]
    _, u = block_norm_forward(x, pre_gain=one, pre_bias=b)
    # |x| is 4096 deviations: the mean is off by a few 2^-24 * 4096
    assert np.abs(u.double().cpu().numpy() - want).max() < 32 * E32 * 4096
    x[1] = 3.0
    x[2, 5] = float("nan")
    _, v = block_norm_forward(x, pre_gain=one, pre_bias=b)
    assert (v[1] == 0.25).all() and torch.equal(v[3], u[3]) and torch.equal(v[0], u[0])
    assert torch.isnan(v[2]).all()


def test_in_place_streams_capture_and_reproducible():
    import torch
    from sketch_attention_compression_b200 import block_norm_backward, block_norm_forward
    x, _ = _make(3001, 128, "bf16", "fp32", 7)
    kw = dict(**_params(x), gate_kind="silu")
    r, u = block_norm_forward(x["x"], x["y"], **kw)
    g = block_norm_backward(r, x["y"], x["dr"], x["du"], **kw)
    again = block_norm_backward(r, x["y"], x["dr"], x["du"], **kw)
    assert all(torch.equal(g[k], again[k]) for k in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r2, u2 = block_norm_forward(x["x"], x["y"], **kw)
        g2 = block_norm_backward(r2, x["y"], x["dr"], x["du"], **kw)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(r, r2) and torch.equal(u, u2) and all(torch.equal(g[k], g2[k]) for k in g)
    inplace = x["x"].clone()
    block_norm_forward(inplace, x["y"], residual_out=inplace, **kw)
    assert torch.equal(inplace, r)


def test_no_rows():
    import torch
    from sketch_attention_compression_b200 import block_norm_backward, block_norm_forward
    x, _ = _make(0, 64, "bf16", "fp32", 7)
    kw = dict(**_params(x), gate_kind="silu")
    r, u = block_norm_forward(x["x"], x["y"], **kw)
    assert r.shape == u.shape == (0, 64)
    g = block_norm_backward(r, x["y"], x["dr"], x["du"], **kw)
    assert g["d_block"].shape == (0, 64)
    for name in ("d_post_gain", "d_post_bias", "d_res_scale", "d_pre_gain", "d_pre_bias"):
        assert (g[name] == 0).all() and g[name].shape == (64,)


def test_refusals():
    import torch
    from sketch_attention_compression_b200 import block_norm_backward, block_norm_forward
    from sketch_attention_compression_b200.binding import SAError
    x, _ = _make(4, 64, "bf16", "fp32", 2)
    args = dict(residual=x["x"], block=x["y"], **_params(x), gate_kind="silu")
    for change, error in (
            (dict(kind="batch"), ValueError), (dict(gate_kind="tanh"), ValueError),
            (dict(block=x["y"][:3]), ValueError), (dict(gate=x["z"].float()), ValueError),
            (dict(pre_gain=x["g2"][:32]), ValueError), (dict(pre_gain=x["g2"].half()), ValueError),
            (dict(eps=0.0), SAError), (dict(residual=x["x"].half()), TypeError),
            (dict(residual=x["x"].cpu()), ValueError), (dict(block=x["y"].t().contiguous().t()), ValueError),
            (dict(pre_gain=None), SAError), (dict(post_gain=None), SAError),
            (dict(residual=x["x"].bfloat16(), block=x["y"].float(), gate=x["z"].float()), SAError),
            (dict(block=None, gate=None), SAError)):
        with pytest.raises(error):
            block_norm_forward(**{**args, **change})
    wide = torch.zeros((2, 8200), device="cuda")
    with pytest.raises(SAError):
        block_norm_forward(wide, pre_gain=torch.ones(8200, device="cuda"))
    with pytest.raises(SAError):
        block_norm_backward(x["x"], x["y"], x["dr"], None, **_params(x))
    with pytest.raises(SAError):
        block_norm_backward(x["x"], x["y"], None, x["du"])
    with pytest.raises(SAError):
        block_norm_backward(x["x"], x["y"], x["dr"], x["du"], **_params(x),
                            workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
