"""Linear attention with values that are not finite, on both scans.

A value that is not finite in v at (row, column) belongs to that column of
its own row and of the rows that the scan reaches after it; everything else
is what the same inputs give with a zero there, within the tolerances of
test_gpu_linear_attention.py (a chunk with such a value may be summed in
another order, with the same roundings)."""

import numpy as np
import pytest

from oracle import linear_attention, linear_attention_grad

pytestmark = pytest.mark.gpu

TOL = {"fp32": 512 * 2.0 ** -24, "bf16": (2 + 1 / 16) * 2.0 ** -8}


def _make(lens, heads, dk, dv, dtype, seed):
    import torch
    gen = torch.Generator().manual_seed(seed)
    n, t = sum(lens), torch.bfloat16 if dtype == "bf16" else torch.float32
    x = {key: torch.randn((n, heads, d), generator=gen).to(t) for key, d in
         (("q", dk), ("k", dk), ("v", dv), ("do", dv))}
    x["g"] = torch.linspace(-0.3, -0.002, heads)
    x["off"] = torch.tensor([0] + lens).cumsum(0)
    return x


def _forward(x, scale=0.125):
    from sketch_attention_compression_b200 import linear_attention_forward, read_device_status
    y = {key: t.cuda() for key, t in x.items()}
    out, state, ws = linear_attention_forward(y["q"], y["k"], y["v"], y["g"], y["off"], scale)
    assert read_device_status(ws) == 0
    return out.double().cpu().numpy(), state.double().cpu().numpy()


def _backward(x, scale=0.125):
    from sketch_attention_compression_b200 import linear_attention_backward, read_device_status
    y = {key: t.cuda() for key, t in x.items()}
    got, ws = linear_attention_backward(y["q"], y["k"], y["v"], y["g"], y["off"], scale, y["do"])
    assert read_device_status(ws) == 0
    return {key: t.double().cpu().numpy() for key, t in got.items()}


def _np(x):
    return {key: t.double().numpy() if key != "off" else t.numpy() for key, t in x.items()}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_single_values_stay_in_their_column(dk, dv, dtype, bad):
    """Values in odd and even rows, in neighbouring columns, in the first and
    the last row of a chunk, and in a short last chunk."""
    x = _make([300], 2, dk, dv, dtype, seed=dk + dv)
    places = [(0, 0, 5), (37, 1, 3), (38, 1, 4), (127, 0, dv - 1), (128, 0, 17), (261, 1, 62), (299, 0, 20)]
    w = _np(x)
    for r, h, c in places:
        x["v"][r, h, c] = bad
        w["v"][r, h, c] = 0.0
    a = {key: np.abs(t) for key, t in w.items()}
    want, _ = linear_attention(w["q"], w["k"], w["v"], w["g"], w["off"], 0.125)
    mag, _ = linear_attention(a["q"], a["k"], a["v"], w["g"], w["off"], 0.125)
    got, state = _forward(x)
    spoiled = np.zeros(got.shape, bool)
    for r, h, c in places:
        spoiled[r:, h, c] = True
        assert not np.isfinite(state[0, h, :, c]).any()
    assert not np.isfinite(got[spoiled]).any()
    good = ~spoiled
    assert np.isfinite(got[good]).all()
    assert (np.abs(got - want)[good] <= TOL[dtype] * mag[good] + 1e-36).all()
    # dk's scan runs from the last row to the first, its columns are those of q
    x = _make([300], 2, dk, dv, dtype, seed=dk + dv)
    w = _np(x)
    x["q"][150, 1, 9] = bad
    w["q"][150, 1, 9] = 0.0
    a = {key: np.abs(t) for key, t in w.items()}
    args = (w["g"], w["off"], 0.125)
    want = linear_attention_grad(w["q"], w["k"], w["v"], *args, w["do"])
    mag = linear_attention_grad(a["q"], a["k"], a["v"], *args, a["do"])
    got = _backward(x)
    spoiled = np.zeros(got["dk"].shape, bool)
    spoiled[:151, 1, 9] = True
    assert not np.isfinite(got["dk"][spoiled]).any()
    good = ~spoiled
    assert (np.abs(got["dk"] - want["dk"])[good] <= TOL[dtype] * mag["dk"][good] + 1e-36).all()
    assert (np.abs(got["dq"] - want["dq"]) <= TOL[dtype] * mag["dq"] + 1e-36).all()
    # dv multiplies q into its weights: every column of the rows up to it
    assert not np.isfinite(got["dv"][:151, 1]).any()
    assert (np.abs(got["dv"] - want["dv"])[151:] <= TOL[dtype] * mag["dv"][151:] + 1e-36).all()


@pytest.mark.parametrize("key", ["k", "v"])
@pytest.mark.parametrize("row", [0, 127, 128, 255])
def test_whole_rows_at_both_ends_of_a_chunk(key, row):
    """A row of NaN or infinities: the rows before it are right, those from it
    on are not finite, and the call does not become much slower."""
    import torch
    for bad in (float("nan"), float("inf")):
        x = _make([256, 40], 2, 128, 128, "bf16", seed=row)
        w = _np(x)
        x[key][row] = bad
        w[key][row] = 0.0
        a = {name: np.abs(t) for name, t in w.items()}
        want, _ = linear_attention(w["q"], w["k"], w["v"], w["g"], w["off"], 0.125)
        mag, _ = linear_attention(a["q"], a["k"], a["v"], w["g"], w["off"], 0.125)
        got, _ = _forward(x)
        ok = np.r_[0:row, 256:296]
        assert (np.abs(got - want)[ok] <= TOL["bf16"] * mag[ok] + 1e-36).all()
        assert not np.isfinite(got[row:256]).any()


@pytest.mark.parametrize("key,row", [("k", 0), ("k", 127), ("v", 0), ("v", 127), ("q", 0),
                                     ("do", 127)])
def test_time_with_rows_that_are_not_finite(key, row):
    """64 users of 512 rows, each with one such row.  The chunk that holds it
    is summed again at some 40 times the time of a chunk: with four chunks a
    user the call may take some ten times as long.  A row's weights taken anew
    for each of its 128 outputs would be 128 times as many."""
    import torch
    from sketch_attention_compression_b200 import linear_attention_backward, linear_attention_forward
    x = _make([512] * 64, 4, 128, 128, "bf16", seed=1)
    y = {name: t.cuda() for name, t in x.items()}
    z = {name: t.clone() for name, t in y.items()}
    z[key].view(64, 512, 4, 128)[:, 128 + row] = float("nan")

    def best(t):
        times = []
        for _ in range(5):
            e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            e[0].record()
            args = (t["q"], t["k"], t["v"], t["g"], t["off"], 0.125)
            linear_attention_forward(*args, max_rows=512)
            linear_attention_backward(*args, t["do"], max_rows=512)
            e[1].record()
            torch.cuda.synchronize()
            times.append(e[0].elapsed_time(e[1]))
        return min(times)

    finite, spoiled = best(y), best(z)
    print(f"{key} {row}: {finite * 1e3:.0f} us, {spoiled * 1e3:.0f} us with NaN")
    assert spoiled <= 30 * finite
