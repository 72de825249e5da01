"""Linear attention, the block norms and gradient clipping used together: one
residual block around causal attention over a ragged batch, trained for a
step, and then served row by row from the state that the prompt left.

The reference is the same block in 64 bits with torch's own differentiation,
evaluated at the bf16 values that the operators pass to each other.  Every
bf16 tensor between two operators is rounded by at most 2^-8 of itself; the
loss gradient passes at most six of them, so a gradient's norm is within
6 * 2^-8 of the reference's plus the operators' own two roundings of 2^-8.
"""

import math

import pytest

pytestmark = pytest.mark.gpu

LENS, H, D = [70, 0, 200, 129, 1], 2, 64
W = H * D
TOL = 8 * 2.0 ** -8


def _setup():
    import torch
    gen = torch.Generator().manual_seed(4)
    n = sum(LENS)

    def draw(*shape, dtype=torch.float32, mul=1.0, add=0.0):
        return (torch.randn(shape, generator=gen) * mul + add).to(dtype).cuda()

    p = dict(x=draw(n, W), g_in=draw(W, mul=0.1, add=1.0), g_post=draw(W, mul=0.1, add=1.0),
             rs=draw(W, mul=0.1, add=0.5), g_out=draw(W, mul=0.1, add=1.0),
             w_qkv=draw(W, 3 * W, dtype=torch.bfloat16, mul=W ** -0.5),
             w_gate=draw(W, W, dtype=torch.bfloat16, mul=W ** -0.5))
    p["g"] = torch.tensor([-0.01, -0.2]).cuda()
    p["off"] = torch.tensor([0] + LENS).cumsum(0).cuda()
    return p, draw(n, W), draw(n, W, dtype=torch.bfloat16)


def _forward(p):
    """(saved tensors, r, u) by the library's operators."""
    import torch
    from sketch_attention_compression_b200 import block_norm_forward, linear_attention_forward
    _, h = block_norm_forward(p["x"], pre_gain=p["g_in"], kind="rms", dtype=torch.bfloat16)
    qkv = (h @ p["w_qkv"]).view(-1, 3, H, D)
    z = h @ p["w_gate"]
    q, k, v = qkv[:, 0], qkv[:, 1], qkv[:, 2]
    y, state, _ = linear_attention_forward(q, k, v, p["g"], p["off"], D ** -0.5, max_rows=max(LENS))
    r, u = block_norm_forward(p["x"], y.view(-1, W), z, post_gain=p["g_post"], res_scale=p["rs"],
                              pre_gain=p["g_out"], kind="rms", gate_kind="silu")
    return dict(h=h, q=q, k=k, v=v, z=z, y=y, state=state), r, u


def _reference(p, s, dr, du):
    """Gradients in 64 bits, through the values the operators saved."""
    import torch
    leaf = {k: p[k].double().clone().requires_grad_() for k in ("x", "g_in", "g_post", "rs", "g_out",
                                                                "w_qkv", "w_gate")}

    def rms(x, gain):
        return gain * x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5)

    def at(value, saved):  # the derivative of `value`, at the saved value
        return value + (saved.double().reshape(value.shape) - value).detach()

    h = at(rms(leaf["x"], leaf["g_in"]), s["h"])
    qkv = h @ leaf["w_qkv"]
    saved = torch.stack([s["q"], s["k"], s["v"]], 1).reshape(qkv.shape)
    q, k, v = at(qkv, saved).view(-1, 3, H, D).unbind(1)
    z = at(h @ leaf["w_gate"], s["z"])
    outs, lo = [], 0
    g = p["g"].double()
    for n in LENS:
        i = torch.arange(n, device="cuda", dtype=torch.float64)
        w = torch.tril(torch.exp(g[:, None, None] * (i[:, None] - i).clamp(min=0)))
        a = torch.einsum("ihd,jhd->hij", q[lo:lo + n], k[lo:lo + n]) * w
        outs.append(torch.einsum("hij,jhd->ihd", a, v[lo:lo + n]) * D ** -0.5)
        lo += n
    y = at(torch.cat(outs).reshape(-1, W), s["y"])
    r = leaf["x"] + leaf["rs"] * z * torch.sigmoid(z) * rms(y, leaf["g_post"])
    u = rms(r, leaf["g_out"])
    loss = (r * dr.double()).sum() + (u * du.double()).sum()
    return dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values())))), r, u


def _backward(p, s, r, dr, du):
    import torch
    from sketch_attention_compression_b200 import block_norm_backward, linear_attention_backward
    out = block_norm_backward(r, s["y"].view(-1, W), dr, du, s["z"], post_gain=p["g_post"],
                              res_scale=p["rs"], pre_gain=p["g_out"], kind="rms", gate_kind="silu")
    att, _ = linear_attention_backward(s["q"], s["k"], s["v"], p["g"], p["off"], D ** -0.5,
                                       out["d_block"].view(-1, H, D), max_rows=max(LENS))
    dqkv = torch.stack([att["dq"], att["dk"], att["dv"]], 1).reshape(-1, 3 * W)
    dh = dqkv @ p["w_qkv"].t() + out["d_gate"] @ p["w_gate"].t()
    first = block_norm_backward(p["x"], None, out["d_residual"], dh, pre_gain=p["g_in"], kind="rms")
    return dict(x=first["d_residual"], g_in=first["d_pre_gain"], g_post=out["d_post_gain"],
                rs=out["d_res_scale"], g_out=out["d_pre_gain"], w_qkv=s["h"].t() @ dqkv,
                w_gate=s["h"].t() @ out["d_gate"])


def test_a_training_step():
    import torch
    from sketch_attention_compression_b200 import clip_grad_norm
    p, dr, du = _setup()
    s, r, u = _forward(p)
    want, r64, u64 = _reference(p, s, dr, du)
    assert (r.double() - r64).norm() <= 2.0 ** -20 * r64.norm()
    assert (u.double() - u64).norm() <= 2.0 ** -8 * u64.norm()
    got = _backward(p, s, r, dr, du)
    for name, g in got.items():
        assert (g.double() - want[name]).norm() <= TOL * want[name].norm(), name
    grads = [got[k].contiguous() for k in got]
    total = math.sqrt(sum(g.double().square().sum().item() for g in grads))
    before = [g.clone() for g in grads]
    norm = clip_grad_norm(grads, 0.5 * total)
    assert abs(norm.item() - total) <= 2.0 ** -20 * total
    for a, b in zip(grads, before):
        assert (a.double() - 0.5 * b.double()).abs().max() <= 2.0 ** -7 * b.double().abs().max()
    # the whole step captured, beside an eager one
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s2, r2, u2 = _forward(p)
        g2 = _backward(p, s2, r2, dr, du)
    graph.replay()
    s3, r3, _ = _forward(p)
    torch.cuda.synchronize()
    assert torch.equal(r2, r) and torch.equal(r3, r) and torch.equal(u2, u)
    assert all(torch.equal(g2[k], b) for k, b in zip(got, before))


def test_a_prompt_then_single_rows():
    """A prompt of all rows but the last three, then those one by one in a
    pool of states, against one pass over everything."""
    import torch
    from sketch_attention_compression_b200 import linear_attention_forward, linear_attention_step
    p, _, _ = _setup()
    s, _, _ = _forward(p)
    lens = torch.tensor(LENS)
    ends = torch.cumsum(lens, 0)
    users = [b for b in range(len(LENS)) if LENS[b] >= 4]
    keep = torch.cat([torch.arange(ends[b] - lens[b], ends[b] - 3) for b in users]).cuda()
    off = torch.tensor([0] + [LENS[b] - 3 for b in users]).cumsum(0).cuda()
    _, state, _ = linear_attention_forward(s["q"][keep], s["k"][keep], s["v"][keep], p["g"], off,
                                           D ** -0.5)
    pool = torch.full((7, H, D, D), 3.0, device="cuda")
    slots = torch.tensor([5, 0, 2], dtype=torch.int64).cuda()
    pool[slots] = state
    for i in range(3):
        rows = torch.tensor([int(ends[b]) - 3 + i for b in users]).cuda()
        out = linear_attention_step(pool, s["q"][rows], s["k"][rows], s["v"][rows], p["g"], D ** -0.5,
                                    slots=slots)
        # the step takes fp32 states, the scan a bf16 copy and bf16 weights
        want = s["y"][rows].double()
        assert (out.double() - want).norm() <= 3 * 2.0 ** -8 * want.norm()
    final = s["state"][users].double()
    assert (pool[slots].double() - final).norm() <= 2.0 ** -18 * final.norm()
    assert (pool[[1, 3, 4, 6]] == 3.0).all()


def test_a_stream_of_its_own():
    """Every operator on a stream that is given, as an object and as a handle,
    while the current stream keeps taking and filling memory: what a call
    allocates is not handed out again before that stream has used it."""
    import torch
    from sketch_attention_compression_b200 import (block_norm_backward, block_norm_forward,
                                                   clip_grad_norm, linear_attention_backward,
                                                   linear_attention_forward, linear_attention_step)
    p, dr, du = _setup()
    s, r, _ = _forward(p)
    state = s["state"].clone()
    big = torch.empty(1 << 26, device="cuda")

    def calls(**kw):
        y, f, _ = linear_attention_forward(s["q"], s["k"], s["v"], p["g"], p["off"], 0.125, **kw)
        g, _ = linear_attention_backward(s["q"], s["k"], s["v"], p["g"], p["off"], 0.125, s["y"], **kw)
        pool = state.clone()
        torch.cuda.synchronize()
        o = linear_attention_step(pool, s["q"][:5], s["k"][:5], s["v"][:5], p["g"], 0.125, **kw)
        r1, u1 = block_norm_forward(p["x"], s["y"].view(-1, W), s["z"], post_gain=p["g_post"],
                                    pre_gain=p["g_out"], gate_kind="silu", **kw)
        b = block_norm_backward(r, s["y"].view(-1, W), dr, du, s["z"], post_gain=p["g_post"],
                                pre_gain=p["g_out"], gate_kind="silu", **kw)
        c = [p["x"].clone(), p["g_in"].clone()]
        torch.cuda.synchronize()
        n = clip_grad_norm(c, 1.0, **kw)
        return [y, f, *g.values(), pool, o, r1, u1, *b.values(), *c, n]

    want = calls()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            big.fill_(1.0)                       # keeps the side stream busy
        got = calls(stream=stream)
        rubbish = [torch.full((n,), 7.0, device="cuda") for n in (1 << 10, 1 << 14, 1 << 18)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del rubbish
