"""Linear attention with a decay per head against its 64-bit recurrence.

Tolerances count roundings against M, the same recurrence over the absolute
values of the inputs (the sum of the magnitudes of all terms of an output):

  fp32 outputs and states  a term passes fewer than 512 fp32 roundings (a dot
      product of <= 128 terms, a chunk of <= 128 rows, the state's sum, and
      one addition per chunk, < 100 chunks here), 2^-24 each: 512 * 2^-24 M.
  bf16 outputs  the weight of a term or the state it comes from is rounded
      once to bf16 (2^-8) and the output once (2^-8): (2 + 1/16) 2^-8 M.

Inputs of few small integers without decay make every intermediate an integer
that bf16 holds, so those runs are compared for equality, row by row.
"""

import numpy as np
import pytest

from oracle import linear_attention, linear_attention_grad, linear_attention_step

pytestmark = pytest.mark.gpu

TOL = {"fp32": 512 * 2.0 ** -24, "bf16": (2 + 1 / 16) * 2.0 ** -8}
DECAYS = [-0.003, 0.0, -0.2, -30.0, -float("inf")]


def _torch_type(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _make(lens, heads, dk, dv, dtype, seed, integers=False):
    """Inputs on the GPU and their values in 64 bits."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    n, b, t = sum(lens), len(lens), _torch_type(dtype)

    def draw(*shape, dtype=t):
        if integers:
            x = torch.randint(-1, 2, shape, generator=gen).float()
            x = x * (torch.rand(shape, generator=gen) < 0.1)
        else:
            x = torch.randn(shape, generator=gen)
        return x.to(dtype)

    x = dict(q=draw(n, heads, dk), k=draw(n, heads, dk), v=draw(n, heads, dv),
             do=draw(n, heads, dv), s0=draw(b, heads, dk, dv, dtype=torch.float32),
             ds=draw(b, heads, dk, dv, dtype=torch.float32))
    decay = [0.0] * heads if integers else [DECAYS[i % len(DECAYS)] for i in range(heads)]
    x["g"] = torch.tensor(decay, dtype=torch.float32)
    x["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int64)
    return {key: v.cuda() for key, v in x.items()}, {key: v.double().numpy() if key != "offsets"
                                                     else v.numpy() for key, v in x.items()}


def _close(got, want, magnitude, tol, what):
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    # 1e-36: results below the smallest normal fp32 are flushed or rounded absolutely
    bad = np.abs(got - want) > tol * magnitude + 1e-36
    assert not bad.any(), f"{what}: {np.argwhere(bad)[:4].tolist()}, " \
        f"{(np.abs(got - want) / (magnitude + 1e-36)).max():.3g} of the magnitude"


def _forward(x, scale, state=True, **kw):
    from sketch_attention_compression_b200 import linear_attention_forward, read_device_status
    out, fin, ws = linear_attention_forward(x["q"], x["k"], x["v"], x["g"], x["offsets"], scale,
                                            initial_state=x["s0"] if state else None, **kw)
    assert read_device_status(ws) == 0
    return out, fin


def _backward(x, scale, state=True, **kw):
    from sketch_attention_compression_b200 import linear_attention_backward, read_device_status
    g, ws = linear_attention_backward(x["q"], x["k"], x["v"], x["g"], x["offsets"], scale, x["do"],
                                      initial_state=x["s0"] if state else None,
                                      d_final_state=x["ds"] if state else None, **kw)
    assert read_device_status(ws) == 0
    return g


def _check(x, w, dtype, scale, state=True, **kw):
    out, fin = _forward(x, scale, state, **kw)
    a = {key: np.abs(val) for key, val in w.items() if key != "g"}
    s0, ds = (w["s0"], w["ds"]) if state else (None, None)
    a0, ad = (a["s0"], a["ds"]) if state else (None, None)
    o, f = linear_attention(w["q"], w["k"], w["v"], w["g"], w["offsets"], scale, s0)
    mo, mf = linear_attention(a["q"], a["k"], a["v"], w["g"], w["offsets"], abs(scale), a0)
    _close(out, o, mo, TOL[dtype], "out")
    _close(fin, f, mf, TOL["fp32"], "final state")
    got = _backward(x, scale, state, **kw)
    args = (w["g"], w["offsets"])
    want = linear_attention_grad(w["q"], w["k"], w["v"], *args, scale, w["do"], s0, ds)
    mag = linear_attention_grad(a["q"], a["k"], a["v"], *args, abs(scale), a["do"], a0, ad)
    for name, val in got.items():
        _close(val, want[name], mag[name], TOL["fp32" if "state" in name else dtype], name)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,heads,dk,dv,state", [
    ([1], 2, 64, 64, True),
    ([17, 0, 63, 64, 65], 3, 64, 128, True),
    ([127, 128, 129], 2, 128, 64, False),
    ([0, 301, 5, 256], 5, 128, 128, True),
    ([0, 0], 2, 64, 64, True),
    ([700, 3, 0, 40], 5, 64, 64, False),   # one long history: split along its rows
    ([2000], 1, 128, 128, True),
])
def test_against_the_recurrence(lens, heads, dk, dv, state, dtype):
    x, w = _make(lens, heads, dk, dv, dtype, seed=sum(lens) + heads)
    _check(x, w, dtype, dk ** -0.5, state)
    if sum(lens) == 2000:
        _check(x, w, dtype, -0.25, state, max_rows=2000)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [[1, 2, 0, 130], [64, 65, 127, 128, 129], [300, 31, 1, 257],
                                  [1900]])
def test_integers_are_exact(lens, dtype):
    import torch
    x, w = _make(lens, 2, 64, 64, dtype, seed=len(lens), integers=True)
    out, fin = _forward(x, 1.0)
    o, f = linear_attention(w["q"], w["k"], w["v"], w["g"], w["offsets"], 1.0, w["s0"])
    assert np.abs(f).max() < 256  # what bf16 holds exactly
    assert torch.equal(out.cpu(), torch.from_numpy(o).to(out.dtype))
    assert np.array_equal(fin.double().cpu().numpy(), f)
    got = _backward(x, 1.0)
    want = linear_attention_grad(w["q"], w["k"], w["v"], w["g"], w["offsets"], 1.0, w["do"],
                                 w["s0"], w["ds"])
    for name, val in got.items():
        assert torch.equal(val.cpu(), torch.from_numpy(want[name]).to(val.dtype)), name


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("users,heads", [(300, 2), (1100, 1)])
def test_more_items_than_sms(users, heads, dtype):
    """Ragged batches of more users than SMs, empty ones among them, also of
    more than are ordered by length."""
    lens = [(i * 37) % 23 for i in range(users)]
    lens[users // 2] = 260
    x, w = _make(lens, heads, 64, 64, dtype, seed=users)
    _check(x, w, dtype, 0.125, max_rows=260)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_split_history_continues_from_its_state(dtype):
    """Two calls, the second from the first one's states, in place."""
    import torch
    lens, cut = [900, 140], [700, 12]
    x, w = _make(lens, 2, 64, 128, dtype, seed=5)
    o, f = linear_attention(w["q"], w["k"], w["v"], w["g"], w["offsets"], 0.125, w["s0"])
    a = {key: np.abs(val) for key, val in w.items() if key != "g"}
    mo, mf = linear_attention(a["q"], a["k"], a["v"], w["g"], w["offsets"], 0.125, a["s0"])
    rows = [np.r_[0:700, 900:912], np.r_[700:900, 912:1040]]
    state, tol = x["s0"].clone(), TOL[dtype]
    for part, n in zip(rows, (cut, [200, 128])):
        idx = torch.from_numpy(part).cuda()
        y = {key: x[key][idx].contiguous() for key in ("q", "k", "v")}
        y |= dict(g=x["g"], s0=state, offsets=torch.tensor([0, n[0], sum(n)]).cuda())
        out, fin = _forward(y, 0.125, final_state=state)
        assert fin.data_ptr() == state.data_ptr()
        _close(out, o[part], mo[part], tol, "out")
    _close(state, f, mf, TOL["fp32"], "state")


def _strided(x, pad_row, pad_head, shift):
    """The same values with other strides and alignment."""
    import torch
    n, h, d = x.shape
    row = h * (d + pad_head) + pad_row
    flat = torch.full((n * row + shift + 64,), float("nan"), dtype=x.dtype, device=x.device)
    y = flat[shift:].as_strided((n, h, d), (row, d + pad_head, 1))
    y.copy_(x)
    return y


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad_row,pad_head,shift", [(8, 0, 8), (64, 16, 0), (3, 0, 0), (0, 1, 0),
                                                    (0, 0, 1)])
def test_strides_and_alignment(pad_row, pad_head, shift, dtype):
    import torch
    x, _ = _make([200, 0, 77], 2, 64, 64, dtype, seed=9)
    want = (*_forward(x, 0.125), *_backward(x, 0.125).values())
    y = dict(x)
    for key in ("q", "k", "v", "do"):
        y[key] = _strided(x[key], pad_row, pad_head, shift)
    got = (*_forward(y, 0.125), *_backward(y, 0.125).values())
    for a, b in zip(got, want):
        # unaligned operands may take the other arithmetic: one more bf16 rounding each way
        tol = 0 if dtype == "fp32" else 5 * 2.0 ** -8
        assert (a.double() - b.double()).abs().max() <= tol * b.double().abs().max() * 2


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_heads_in_any_layout(dtype):
    """q, k, v as slices of one fused projection, and head-major storage."""
    import torch
    x, w = _make([150, 20], 3, 64, 64, dtype, seed=10)
    fused = torch.cat([x["q"], x["k"], x["v"]], dim=2)
    y = dict(x, q=fused[..., :64], k=fused[..., 64:128], v=fused[..., 128:])
    _check(y, w, dtype, 0.125)
    z = dict(x)
    for key in ("q", "k", "v", "do"):
        z[key] = x[key].transpose(0, 1).contiguous().transpose(0, 1)
    _check(z, w, dtype, 0.125)


def _same(a, b, magnitude, dtype, what):
    """fp32: equal.  bf16: both within their tolerance of the same value (a
    chunk that holds a value that is not finite may be summed another way)."""
    if dtype == "fp32":
        assert (a == b).all(), what
    else:
        _close(a, b.double().cpu().numpy(), magnitude, 2 * TOL["bf16"], what)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_of_nobody_and_later_rows_do_not_matter(dtype):
    """Rows behind the last user are left as they were, and neither they nor
    a row's own future reach its output, whatever they hold."""
    import torch
    lens = [150, 60]
    x, w = _make(lens, 2, 64, 64, dtype, seed=11)
    a = {key: np.abs(val) for key, val in w.items() if key != "g"}
    mo, _ = linear_attention(a["q"], a["k"], a["v"], w["g"], w["offsets"], 0.125, a["s0"])
    mag = linear_attention_grad(a["q"], a["k"], a["v"], w["g"], w["offsets"], 0.125, a["do"],
                                a["s0"], a["ds"])
    want, fin = _forward(x, 0.125)
    y = {key: (torch.cat([x[key], torch.full_like(x[key][:50], float("nan"))])
               if key in ("q", "k", "v", "do") else x[key]) for key in x}
    out = torch.full((260, 2, 64), 7.0, dtype=x["q"].dtype, device="cuda")
    got, fin2 = _forward(y, 0.125, out=out)
    assert torch.equal(got[:210], want) and torch.equal(fin, fin2)
    assert (got[210:] == 7).all()
    g1, g2 = _backward(x, 0.125), _backward(y, 0.125)
    for name in ("dq", "dk", "dv"):
        assert torch.equal(g1[name], g2[name][:210]), name
    assert torch.equal(g1["d_initial_state"], g2["d_initial_state"])
    # the future: row 100 of user 0 and row 170 (user 1) are poisoned
    for key in ("k", "v"):
        for bad in (float("nan"), float("inf")):
            z = {n: t.clone() for n, t in x.items()}
            z[key][100] = bad
            z[key][170] = bad
            got, _ = _forward(z, 0.125)
            _same(got[:100], want[:100], mo[:100], dtype, (key, bad))
            _same(got[150:170], want[150:170], mo[150:170], dtype, (key, bad))
            assert not torch.isfinite(got[100].float()).any()
    # the gradients' scans: dq sees k and v up to its row, dk and dv see q and do from theirs on
    for key in ("k", "v"):
        z = {n: t.clone() for n, t in x.items()}
        z[key][100] = float("nan")
        got = _backward(z, 0.125)
        _same(got["dq"][:100], g1["dq"][:100], mag["dq"][:100], dtype, key)
        assert not torch.isfinite(got["dq"][100].float()).any()
    for key in ("q", "do"):
        z = {n: t.clone() for n, t in x.items()}
        z[key][100] = float("nan")
        got = _backward(z, 0.125)
        for name in ("dk", "dv"):
            _same(got[name][101:], g1[name][101:], mag[name][101:], dtype, (key, name))


def test_flags():
    import torch
    from sketch_attention_compression_b200 import linear_attention_forward, read_device_status
    x, _ = _make([100, 20], 2, 64, 64, "bf16", seed=12)
    for offsets, decay, flag in (([0, 100, 121], 0.0, 4), ([1, 100, 120], 0.0, 1),
                                 ([0, 100, 90], 0.0, 2), ([0, 100, 120], 0.5, 64),
                                 ([0, 100, 120], float("nan"), 64), ([0, 50, 110], 0.0, 0)):
        o = torch.tensor(offsets, dtype=torch.int64).cuda()
        g = torch.tensor([-0.1, decay]).cuda()
        _, _, ws = linear_attention_forward(x["q"], x["k"], x["v"], g, o, 0.125)
        assert read_device_status(ws) == flag, (offsets, decay)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_reproducible_and_captured(dtype):
    """The same call twice, on another stream, and as a replayed graph beside
    an eager call of the same inputs."""
    import torch
    x, _ = _make([900, 130, 0, 33], 2, 64, 64, dtype, seed=13)
    want = (*_forward(x, 0.125), *_backward(x, 0.125).values())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    from sketch_attention_compression_b200 import (linear_attention_backward,
                                                   linear_attention_forward)
    args = (x["q"], x["k"], x["v"], x["g"], x["offsets"], 0.125)
    with torch.cuda.stream(s):
        again = (*_forward(x, 0.125), *_backward(x, 0.125).values())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, f, _ = linear_attention_forward(*args, initial_state=x["s0"])
        g, _ = linear_attention_backward(*args, x["do"], initial_state=x["s0"],
                                         d_final_state=x["ds"])
    for _ in range(2):
        o.zero_()
        g["dk"].zero_()
        graph.replay()
        eager = _forward(x, 0.125)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (o, f, *g.values())))
        assert torch.equal(eager[0], want[0])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("batch,heads,dk,dv", [(1, 2, 64, 64), (3, 1, 1, 4), (7, 3, 96, 100),
                                               (40, 8, 128, 128), (300, 1, 37, 256),
                                               (2, 2, 256, 8)])
def test_step(batch, heads, dk, dv, dtype):
    x, w = _make([1] * batch, heads, dk, dv, dtype, seed=batch + dk)
    from sketch_attention_compression_b200 import linear_attention_step
    state = x["s0"].clone()
    out = linear_attention_step(state, x["q"], x["k"], x["v"], x["g"], 0.3)
    o, s = linear_attention_step_oracle(w, 0.3)
    a = {key: np.abs(val) for key, val in w.items() if key != "g"} | {"g": w["g"]}
    mo, ms = linear_attention_step_oracle(a, 0.3)
    _close(out, o, mo, TOL["fp32"] if dtype == "fp32" else TOL["bf16"], "out")
    _close(state, s, ms, 4 * 2.0 ** -24, "state")


def linear_attention_step_oracle(w, scale, slots=None):
    return linear_attention_step(w["s0"], w["q"], w["k"], w["v"], w["g"], scale, slots)


def test_step_slots():
    import torch
    from sketch_attention_compression_b200 import linear_attention_step
    x, w = _make([1] * 6, 2, 64, 64, "fp32", seed=21)
    state = x["s0"].clone()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([4, -1, 0, 5], dtype=torch.int64).cuda()
    args = (x["q"][:4], x["k"][:4], x["v"][:4], x["g"], 0.5)
    out = linear_attention_step(state, *args, slots=slots, device_flags=flags)
    w4 = {key: val[:4] if key in "qkv" else val for key, val in w.items()}
    o, s = linear_attention_step_oracle(w4, 0.5, [4, -1, 0, 5])
    assert flags.item() == 0 and (out[1] == 0).all()
    np.testing.assert_allclose(out.double().cpu().numpy(), o, rtol=1e-4, atol=1e-4)
    np.testing.assert_allclose(state.double().cpu().numpy(), s, rtol=1e-6, atol=1e-6)
    for i in (1, 2, 3):
        assert torch.equal(state[i], x["s0"][i])
    # a slot twice, and one past the pool: the first entry is taken, the others are refused
    state = x["s0"].clone()
    out = linear_attention_step(state, *args, slots=torch.tensor([3, 3, 6, 3]).cuda(),
                                device_flags=flags)
    assert flags.item() == 128 and (out[1:] == 0).all()
    o, s = linear_attention_step_oracle(w4, 0.5, [3, -1, -1, -1])
    np.testing.assert_allclose(state.double().cpu().numpy(), s, rtol=1e-6, atol=1e-6)
    assert torch.equal(state[:3], x["s0"][:3])


def test_long_history_keeps_its_sums():
    """20000 rows of one head with a horizon of 4096: the state, whose sum is
    32 chunks long and more, against the recurrence."""
    import torch
    for dtype in ("bf16", "fp32"):
        x, w = _make([20000], 1, 64, 64, dtype, seed=31)
        x["g"][0] = float(np.log1p(-2.0 ** -12))
        w["g"] = x["g"].double().cpu().numpy()
        _, fin = _forward(x, 0.125)
        _, f = linear_attention(w["q"], w["k"], w["v"], w["g"], w["offsets"], 0.125, w["s0"])
        err = np.linalg.norm(fin.double().cpu().numpy() - f) / np.linalg.norm(f)
        # The decay of a chunk is kept to 2^-47, the sum of a chunk to some
        # 2^-24 each way, and 4096 / 64 chunks add one rounding each, in
        # random directions: sqrt(64) * 2^-24 and a margin of two.
        assert err < 16 * 2.0 ** -24, err
        torch.cuda.empty_cache()


def test_refusals():
    import torch
    from sketch_attention_compression_b200 import (linear_attention_backward,
                                                   linear_attention_forward,
                                                   linear_attention_step)
    from sketch_attention_compression_b200.binding import SAError
    x, _ = _make([10], 2, 64, 64, "bf16", seed=1)
    args = dict(q=x["q"], k=x["k"], v=x["v"], log_decay=x["g"], offsets=x["offsets"], scale=0.1)
    for change, error in (
            (dict(k=x["k"].float()), TypeError), (dict(k=x["k"][:9]), ValueError),
            (dict(q=x["q"].cpu()), ValueError), (dict(offsets=x["offsets"].int()), TypeError),
            (dict(log_decay=x["g"].double()), ValueError), (dict(scale=float("nan")), SAError),
            (dict(scale=0.0), SAError), (dict(v=x["v"][..., :40].contiguous()), SAError),
            (dict(v=x["v"].transpose(1, 2)), ValueError), (dict(max_rows=-1), SAError),
            (dict(q=x["q"][:, :1].expand(10, 2, 64)), SAError),
            (dict(initial_state=x["s0"][:, :, :, :32]), ValueError),
            (dict(initial_state=x["s0"].bfloat16()), ValueError),
            (dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), SAError)):
        with pytest.raises(error):
            linear_attention_forward(**{**args, **change})
        d_out = x["do"][..., :change["v"].shape[2]] if "v" in change else x["do"]
        with pytest.raises(error):
            linear_attention_backward(**{**args, **change}, d_out=d_out)
    state = x["s0"]
    step = dict(state=state, q=x["q"][:1], k=x["k"][:1], v=x["v"][:1], log_decay=x["g"], scale=1.0)
    for change, error in ((dict(state=state.bfloat16()), ValueError), (dict(state=state[0]), ValueError),
                          (dict(v=x["v"][:1, :, :6], state=state[..., :6].contiguous()), SAError), (dict(k=x["k"][:2]), ValueError),
                          (dict(slots=torch.zeros(1, dtype=torch.int32, device="cuda")), ValueError),
                          (dict(state=state[:0]), SAError)):
        with pytest.raises(error):
            linear_attention_step(**{**step, **change})
