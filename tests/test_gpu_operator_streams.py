"""Operators on a stream that is given: what a call allocates is neither
memory that work queued on the current stream still uses, nor handed out
again while the given stream, or the current one, uses it.  Addresses are compared, so a wrong
allocation shows whether or not two kernels happen to meet in it."""

import pytest

pytestmark = pytest.mark.gpu

LENS, H, D = [300, 0, 129], 2, 64
W, N = H * D, 429
BUSY = 100_000_000  # cycles of one idle kernel: some 50 ms


def _inputs():
    import torch
    gen = torch.Generator().manual_seed(7)

    def draw(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen).to(dtype).cuda()

    f32 = torch.float32
    return dict(q=draw(N, H, D), k=draw(N, H, D), v=draw(N, H, D), do=draw(N, H, D),
                s0=draw(3, H, D, D, dtype=f32), g=torch.tensor([-0.01, -0.3]).cuda(),
                off=torch.tensor([0, 300, 300, 429]).cuda(), x=draw(N, W, dtype=f32), y=draw(N, W),
                z=draw(N, W), dr=draw(N, W, dtype=f32), du=draw(N, W), gain=draw(W, dtype=f32),
                grads=[draw(1000, 77), draw(5, dtype=f32)])


def _calls():
    import sketch_attention_compression_b200 as sa
    norm = lambda i: dict(post_gain=i["gain"], pre_gain=i["gain"], gate_kind="silu")  # noqa: E731
    att = lambda i: (i["q"], i["k"], i["v"], i["g"], i["off"], 0.125)                 # noqa: E731
    return dict(
        forward=lambda i, s: sa.linear_attention_forward(*att(i), initial_state=i["s0"], stream=s)[:2],
        backward=lambda i, s: list(sa.linear_attention_backward(
            *att(i), i["do"], initial_state=i["s0"], stream=s)[0].values()),
        step=lambda i, s: (sa.linear_attention_step(
            i["s0"], i["q"][:3], i["k"][:3], i["v"][:3], i["g"], 0.125, stream=s), i["s0"]),
        norm_forward=lambda i, s: sa.block_norm_forward(i["x"], i["y"], i["z"], stream=s, **norm(i)),
        norm_backward=lambda i, s: list(sa.block_norm_backward(
            i["x"], i["y"], i["dr"], i["du"], i["z"], stream=s, **norm(i)).values()),
        norm=lambda i, s: [sa.grad_norm(i["grads"], stream=s)],
        clip=lambda i, s: [sa.clip_grad_norm(i["grads"], 1.0, stream=s), *i["grads"]])


def _span(t):
    return t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()


def _apart(spans, others):
    return all(a1 <= b0 or b1 <= a0 for a0, a1 in spans for b0, b1 in others)


@pytest.mark.parametrize("name", ["forward", "backward", "step", "norm_forward", "norm_backward", "norm",
                                  "clip"])
@pytest.mark.parametrize("as_handle", [False, True])
def test_memory_of_a_call_on_another_stream(name, as_handle, monkeypatch):
    _memory_of_a_call(_calls()[name], _inputs, as_handle, monkeypatch)


def _memory_of_a_call(call, make, as_handle, monkeypatch):
    import torch
    from sketch_attention_compression_b200 import binding
    taken, used_on = [], binding._used_on

    def spy(stream, *tensors):
        taken.extend(t for t in tensors if t is not None and t.numel() > 0)
        used_on(stream, *tensors)

    monkeypatch.setattr(binding, "_used_on", spy)
    want = [t.clone() for t in call(make(), None)]
    sizes = [(t.shape, t.dtype) for t in taken]
    taken.clear()
    first, second = make(), make()
    side = torch.cuda.Stream()
    given = side.cuda_stream if as_handle else side
    # Memory that is free again on the current stream, and still read there.
    held = [torch.full(s, 7, dtype=t, device="cuda") for s, t in sizes for _ in range(3)]
    copies = [torch.empty_like(t) for t in held]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for c, t in zip(copies, held):
        c.copy_(t)
    spans = [_span(t) for t in held]
    del held, t
    got = call(first, given)
    assert _apart(spans, [_span(t) for t in taken])
    torch.cuda.synchronize()
    assert all(bool((c == 7).all()) for c in copies)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # Memory that is dropped while the given stream has yet to use it.
    del got
    taken.clear()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = [t.data_ptr() for t in call(second, given)]
    spans = [_span(t) for t in taken]
    taken.clear()
    new = [torch.full(s, 9, dtype=t, device="cuda") for s, t in sizes for _ in range(3)]
    assert not side.query() and len(got) == len(want)
    assert _apart(spans, [_span(t) for t in new])
    torch.cuda.synchronize()
    assert all(bool((t == 9).all()) for t in new)
    # Results that the current stream reads, and that are dropped meanwhile.
    third, fourth = make(), make()
    torch.cuda.synchronize()
    got = call(third, given)
    side.synchronize()
    spans = [_span(t) for t in taken]
    copies = [torch.empty_like(t) for t in got]
    torch.cuda._sleep(BUSY)
    for c, t in zip(copies, got):
        c.copy_(t)
    del got, t
    taken.clear()
    got = call(fourth, given)
    assert _apart(spans, [_span(t) for t in taken])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_captured_call_on_a_forked_stream():
    """A stream that joins a capture: its outputs come from the graph's memory."""
    import torch
    call, i = _calls()["forward"], _inputs()
    want = [t.clone() for t in call(i, None)]
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(i, side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        got[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def _layer_inputs():
    import torch
    from sketch_attention_compression_b200 import ActionFusion, RefineParams, SketchQuery, WidthAdapter
    from synthetic import action_params, action_types, refine_params, upstream_gradients
    from synthetic.workloads import make_inputs
    i = make_inputs([700, 0, 129], d=128, k=64, dtype="bf16", seed=97)
    layer, act = refine_params(128, 256, seed=96), action_params(128, 32, 128, 4, seed=98)

    def f32(a):
        return torch.from_numpy(a).float().cuda()

    def bf16(a):
        return f32(a).to(torch.bfloat16)

    G, g = upstream_gradients(3, 64, 128, seed=95)
    names = ("W1", "W3", "W2", "gamma1", "beta1", "gamma2", "beta2")
    return dict(X=bf16(i["X"]), host_offsets=i["offsets"], off=torch.from_numpy(i["offsets"]).cuda(),
                q=SketchQuery(bf16(i["P"]), bf16(i["W_Q"]), bf16(i["W_K"]), i["scale"]),
                Q=f32(i["P"]).expand(3, 64, 128).contiguous(), P=f32(i["P"]), WQ=f32(i["W_Q"]),
                WK=f32(i["W_K"]), G=f32(G), gm=f32(g), sketch=f32(G), mass=f32(g).abs() + 1.0,
                params=RefineParams(*(f32(layer[n]) for n in names)),
                adapter=WidthAdapter(torch.full((128, 256), 0.125, device="cuda")),
                action=ActionFusion(*(f32(act[n]) for n in ("W1", "W3", "W2", "table"))),
                types=torch.from_numpy(action_types(len(i["X"]), 4, seed=97)).cuda())


def _layer_calls():
    from sketch_attention_compression_b200 import (SketchCache, mass_normalise, refine_layer_forward,
                                                   refine_stack_forward)
    keys = [(b, 1, 100, 7) for b in range(3)]

    def cached(i, s):
        i["cache"] = SketchCache(64, 128, capacity=4, ttl=60.0)
        return i["cache"].forward(i["q"], keys, 0.0, i["X"], i["host_offsets"], stream=s)[:2]

    return dict(
        sketch=lambda i, s: i["q"].forward(i["X"], i["off"], stream=s),
        user_queries=lambda i, s: i["q"].forward_user_queries(i["Q"], i["X"], i["off"], stream=s),
        noalloc=lambda i, s: i["q"].forward_noalloc(i["X"], i["off"], stream=s),
        backward=lambda i, s: list(i["q"].backward(
            i["X"], i["off"], i["G"], i["gm"], P_f32=i["P"], W_Q_f32=i["WQ"], W_K_f32=i["WK"],
            stream=s)[0].values()),
        update=lambda i, s: [i["params"].update(i["Q"], i["sketch"], i["mass"], stream=s)],
        layer=lambda i, s: [refine_layer_forward(i["q"], i["params"], i["X"], i["off"], P_f32=i["P"],
                                                 stream=s)[0]],
        stack=lambda i, s: [refine_stack_forward([i["q"]] * 2, [i["params"]] * 2, i["P"], i["X"],
                                                 i["off"], stream=s)[0]],
        normalise=lambda i, s: [mass_normalise(i["sketch"], i["mass"], stream=s)],
        cached=cached,
        adapter=lambda i, s: [i["adapter"].forward(i["sketch"].view(-1, 128), stream=s)],
        fuse=lambda i, s: [i["action"].fuse(i["X"], i["types"], stream=s)],
        action_sketch=lambda i, s: i["action"].sketch_forward(i["q"], i["X"], i["types"], i["off"],
                                                              stream=s)[:2])


@pytest.mark.parametrize("name", ["sketch", "user_queries", "noalloc", "backward", "update", "layer",
                                  "stack", "normalise", "cached", "adapter", "fuse", "action_sketch"])
def test_memory_of_a_layer_call_on_another_stream(name, monkeypatch):
    _memory_of_a_call(_layer_calls()[name], _layer_inputs, False, monkeypatch)
