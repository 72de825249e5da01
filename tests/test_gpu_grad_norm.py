"""The global gradient norm and clipping against 64 bits.

Squares are added eight at a time in fp32 (8 roundings of 2^-24, all terms
positive) and then in fp64: the norm is within 4.5 * 2^-24 of itself, plus
one rounding to fp32; a scaled value passes the factor's rounding, the norm's
error and one more rounding to its type.
"""

import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

E32, E16 = 2.0 ** -24, 2.0 ** -8


def _tensors(shapes, dtypes, seed, mul=0.02):
    import torch
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=gen) * mul).to(torch.bfloat16 if t == "bf16" else torch.float32)
            .cuda() for s, t in zip(shapes, dtypes)]


def _norm64(grads):
    return math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))


def _check(grads, max_norm, **kw):
    import torch
    from sketch_attention_compression_b200 import clip_grad_norm, grad_norm
    want = _norm64(grads)
    got = grad_norm(grads, **kw)
    assert abs(got.item() - want) <= 6 * E32 * want
    before = [g.clone() for g in grads]
    out = [torch.full_like(g, 7.0) for g in grads]
    n1 = clip_grad_norm(grads, max_norm, out=out, **kw)
    assert torch.equal(n1, got) and all(torch.equal(a, b) for a, b in zip(before, grads))
    mul = min(1.0, max_norm / (want + 1e-6))
    for o, g in zip(out, grads):
        w = g.double() * mul
        tol = (8 * E32 + (E16 if g.dtype == torch.bfloat16 else E32)) * w.abs() + 1e-38
        assert ((o.double() - w).abs() <= tol).all()
    n2 = clip_grad_norm(grads, max_norm, **kw)
    assert torch.equal(n2, got) and all(torch.equal(a, b) for a, b in zip(grads, out))


@pytest.mark.parametrize("shapes,dtypes", [
    ([(1,)], ["fp32"]), ([(1,), (3,), (8,), (2047,), (2048,), (2049,)], ["bf16"] * 6),
    ([(128, 512), (0, 5), (77,), (1000, 129)], ["fp32", "fp32", "bf16", "bf16"]),
    ([(300, 1025)], ["bf16"]), ([(64,)] * 60 + [(4096, 300)], ["fp32"] * 30 + ["bf16"] * 31),
    ([(17,)] * 2000, ["bf16", "fp32"] * 1000), ([()], ["fp32"])])
@pytest.mark.parametrize("max_norm", [0.5, 1e6, 0.0])
def test_norm_and_clip(shapes, dtypes, max_norm):
    _check(_tensors(shapes, dtypes, seed=len(shapes)), max_norm)


def test_unaligned_views():
    flat = _tensors([(100000,)], ["bf16"], 3)[0]
    _check([flat[1:5000], flat[5001:5004], flat[5008:90001], flat[90003:]], 0.1)


def test_range():
    """Gradients near both ends of fp32: no overflow, no loss."""
    import torch
    from sketch_attention_compression_b200 import grad_norm
    for mul in (1e-38, 1e-30, 1e-20, 1e15, 1e18, 1e30, 1e37):
        g = [torch.full((1000,), mul, device="cuda"), torch.full((24,), mul, device="cuda")]
        want = _norm64(g)
        if want < 3e38:
            assert abs(grad_norm(g).item() - want) <= 6 * E32 * want, mul
    assert grad_norm([torch.zeros(10, device="cuda")]).item() == 0.0


def test_not_finite_leaves_the_values():
    import torch
    from sketch_attention_compression_b200 import clip_grad_norm
    for bad in (float("nan"), float("inf")):
        g = _tensors([(5000,), (100,)], ["bf16", "fp32"], 5)
        g[1][7] = bad
        before = [x.clone() for x in g]
        n = clip_grad_norm(g, 0.01)
        assert not math.isfinite(n.item())
        assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(g, before))


def test_reproducible_streams_and_capture():
    import torch
    from sketch_attention_compression_b200 import clip_grad_norm
    grads = _tensors([(1 << 20,), (333,), (100, 1001)], ["bf16", "fp32", "fp32"], 8)
    out = [torch.empty_like(g) for g in grads]
    n = clip_grad_norm(grads, 0.3, out=out)
    want = [o.clone() for o in out]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        n2 = clip_grad_norm(grads, 0.3, out=out)
    torch.cuda.synchronize()
    assert torch.equal(n, n2) and all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n3 = clip_grad_norm(grads, 0.3, out=out)
    grads[1].mul_(100.0)  # the graph reads the values of its replay
    other = [torch.empty_like(g) for g in grads]
    for _ in range(2):
        graph.replay()
        n4 = clip_grad_norm(grads, 0.3, out=other)
    torch.cuda.synchronize()
    assert torch.equal(n3, n4) and not torch.equal(n3, n)
    assert all(torch.equal(a, b) for a, b in zip(out, other))


def test_no_gradients():
    import torch
    from sketch_attention_compression_b200 import clip_grad_norm, grad_norm
    assert grad_norm([], device="cuda").item() == 0.0
    assert clip_grad_norm([torch.empty(0, device="cuda")], 1.0).item() == 0.0


def test_refusals():
    import torch
    from sketch_attention_compression_b200 import clip_grad_norm, grad_norm
    from sketch_attention_compression_b200.binding import SAError
    a, b = _tensors([(64, 32), (100,)], ["fp32", "bf16"], 1)
    with pytest.raises(ValueError):
        grad_norm([a.t()])
    with pytest.raises(TypeError):
        grad_norm([a.half()])
    with pytest.raises(ValueError):
        grad_norm([a.cpu()])
    with pytest.raises(ValueError):
        grad_norm([])
    for bad in (-1.0, float("nan"), float("inf")):
        with pytest.raises(SAError):
            clip_grad_norm([a], bad)
    with pytest.raises(SAError):
        clip_grad_norm([a, b, a], 1.0)              # a tensor twice
    with pytest.raises(SAError):
        clip_grad_norm([a, a[3]], 1.0)              # overlapping views
    with pytest.raises(SAError):
        clip_grad_norm([b[:50]], 1.0, out=[b[1:51]])
    with pytest.raises(ValueError):
        clip_grad_norm([a, b], 1.0, out=[a])
    with pytest.raises(SAError):
        grad_norm([a], workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert abs(grad_norm([a, a]).item() - np.sqrt(2) * _norm64([a])) < 1e-5  # reading twice is fine
