"""Linear attention where the decay matters, in relative 2-norms, and the
forward that returns no state.

With random inputs the terms of an output have random signs, so its norm is
near R, the root of the sum of their squares (the same recurrence over the
squared inputs), and its error's is near a rounding times R.  bf16: the weight
(or state) of a term and the output are rounded by at most 2^-8 each, at most
2^-8 / sqrt(3) in the mean of squares: sqrt(2 / 3) 2^-8, and 2^-8 is asked
for.  fp32 (and the states of bf16 calls): a sum of some 200 roundings in
random directions is off by sqrt(200 / 3) 2^-24 R; 32 * 2^-24 is asked for.  A
power of the decay that is off by one row would show as 5 % and more.

Why R and not the output's own norm: a user of one row without a state has
the output scale (q . k) v.  The dot product's rounding errors go with the
magnitudes of its products, sqrt(d_k) where these are of order 1, while q . k
itself can be any fraction of that: for one such row here (0.186 against
10.3) it is 2 % of it, and its error 4e-6 of itself, but 7e-8 of R."""

import numpy as np
import pytest

from oracle import linear_attention, linear_attention_grad

pytestmark = pytest.mark.gpu

TOL = {"bf16": 2.0 ** -8, "fp32": 32 * 2.0 ** -24}


def _make(lens, decays, dk, dv, dtype):
    import torch
    gen = torch.Generator().manual_seed(dk + 3 * dv + len(lens))
    n, b, h = sum(lens), len(lens), len(decays)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = {key: torch.randn((n, h, d), generator=gen).to(t) for key, d in
         (("q", dk), ("k", dk), ("v", dv), ("do", dv))}
    x |= {key: torch.randn((b, h, dk, dv), generator=gen) for key in ("s0", "ds")}
    x |= dict(g=torch.tensor(decays), off=torch.tensor([0] + lens).cumsum(0))
    return ({key: t.cuda() for key, t in x.items()},
            {key: t.double().numpy() if key != "off" else t.numpy() for key, t in x.items()})


def _rows_close(got, want, squares, off, tol, what):
    """Per user and head: short users do not hide behind long ones."""
    got = got.double().cpu().numpy()
    for b in range(len(off) - 1):
        for h in range(got.shape[1]):
            a, w, r = (t[off[b]:off[b + 1], h] for t in (got, want, np.sqrt(squares)))
            size = max(np.linalg.norm(w), np.linalg.norm(r))
            assert np.linalg.norm(a - w) <= tol * size, (what, b, h)


def _squares(w):
    """The inputs whose recurrence is the sum of the squares of all terms."""
    return {key: t if key == "off" else 2 * t if key == "g" else t * t for key, t in w.items()}


SHAPES = [([300, 1, 0, 129, 128], [-0.2, -0.5]), ([300, 1, 0, 129, 128], [-0.7]), ([1500], [-0.05])]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("lens,decays", SHAPES)
def test_strong_decays_in_every_head(lens, decays, dk, dv, dtype):
    from sketch_attention_compression_b200 import linear_attention_backward, linear_attention_forward
    x, w = _make(lens, decays, dk, dv, dtype)
    args, kw = (x["q"], x["k"], x["v"], x["g"], x["off"], 0.125), dict(max_rows=max(lens))
    out, state, _ = linear_attention_forward(*args, initial_state=x["s0"], **kw)
    o, s = linear_attention(w["q"], w["k"], w["v"], w["g"], w["off"], 0.125, w["s0"])
    y = _squares(w)
    ro, rs = linear_attention(y["q"], y["k"], y["v"], y["g"], w["off"], 0.125 ** 2, y["s0"])
    _rows_close(out, o, ro, w["off"], TOL[dtype], "out")
    users = np.arange(len(lens) + 1)
    _rows_close(state, s, rs, users, TOL["fp32"], "state")
    got, _ = linear_attention_backward(*args, x["do"], initial_state=x["s0"], d_final_state=x["ds"], **kw)
    want = linear_attention_grad(w["q"], w["k"], w["v"], w["g"], w["off"], 0.125, w["do"], w["s0"], w["ds"])
    r = linear_attention_grad(y["q"], y["k"], y["v"], y["g"], w["off"], 0.125 ** 2, y["do"], y["s0"],
                              y["ds"])
    for name in ("dq", "dk", "dv"):
        _rows_close(got[name], want[name], r[name], w["off"], TOL[dtype], name)
    name = "d_initial_state"
    _rows_close(got[name], want[name], r[name], users, TOL["fp32"], name)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("lens,decays", SHAPES + [([700, 3, 0, 40], [-0.003, -0.2, 0.0, -30.0])])
@pytest.mark.parametrize("start", [False, True])
def test_a_forward_without_a_final_state(lens, decays, dk, dv, dtype, start):
    """The C call with final_state NULL: the products of the state have fewer parts."""
    import torch
    from sketch_attention_compression_b200 import binding, read_device_status
    lib = binding.load_library()
    x, w = _make(lens, decays, dk, dv, dtype)
    n, h, b = sum(lens), len(decays), len(lens)
    ws = torch.empty(lib.sa_workspace_bytes_linear_attention(h, dk, dv, b, n, max(lens)),
                     dtype=torch.uint8, device="cuda")
    out = torch.full_like(x["v"], 7.0)
    qkv = [a for key, d in (("q", dk), ("k", dk), ("v", dv)) for a in (x[key].data_ptr(), h * d, d)]
    assert lib.sa_linear_attention_forward(
        *qkv, x["g"].data_ptr(), x["off"].data_ptr(), b, n, max(lens), h, dk, dv,
        binding.SA_BF16 if dtype == "bf16" else binding.SA_FP32, 0.125,
        x["s0"].data_ptr() if start else None, out.data_ptr(), None, ws.data_ptr(), ws.numel(),
        torch.cuda.current_stream().cuda_stream) == binding.SA_OK
    assert read_device_status(ws) == 0
    o, _ = linear_attention(w["q"], w["k"], w["v"], w["g"], w["off"], 0.125, w["s0"] if start else None)
    y = _squares(w)
    ro, _ = linear_attention(y["q"], y["k"], y["v"], y["g"], w["off"], 0.125 ** 2,
                             y["s0"] if start else None)
    _rows_close(out, o, ro, w["off"], TOL[dtype], "out")
