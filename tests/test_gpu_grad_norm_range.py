"""Clipping at the ends of the range of fp32.  Tolerances as in
test_gpu_grad_norm.py: a scaled value is within 9 roundings of 2^-24 of
itself (2^-8 more for bf16) and of the spacing of the smallest results."""

import math

import pytest

pytestmark = pytest.mark.gpu

E32, E16 = 2.0 ** -24, 2.0 ** -8


def _full(value, *shapes, dtype="float32"):
    import torch
    return [torch.full(s, value, dtype=getattr(torch, dtype), device="cuda") for s in shapes]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("value,count", [(3e38, 1024), (3e38, 2), (2.5e38, 100000)])
def test_a_norm_beyond_fp32_leaves_the_values(value, count, dtype):
    """Finite values whose norm is not: the norm that is told decides."""
    import torch
    from sketch_attention_compression_b200 import clip_grad_norm, grad_norm
    g = _full(value, (count - 1,), (1,), dtype=dtype)
    before = [x.clone() for x in g]
    out = [torch.zeros_like(x) for x in g]
    assert math.isinf(grad_norm(g).item())
    assert math.isinf(clip_grad_norm(g, 1.0, out=out).item())
    assert all(torch.equal(a, b) for a, b in zip(out, before))
    assert math.isinf(clip_grad_norm(g, 1.0).item())
    assert all(torch.equal(a, b) for a, b in zip(g, before))


def test_the_largest_norm_in_fp32_still_clips():
    import torch
    from sketch_attention_compression_b200 import clip_grad_norm
    g = _full(1.5e38, (4,))  # norm 3e38
    norm = clip_grad_norm(g, 8.0)
    assert abs(norm.item() - 3e38) <= 4 * E32 * 3e38
    assert (g[0].double() - 4.0).abs().max() <= 9 * E32 * 4.0


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("value,max_norm", [(1e37, 1.0), (1e37, 1e-3), (1e36, 1e-5), (3e35, 1e-38),
                                            (1e30, 1e-30), (1e30, 1e-20), (1.0, 1e-39)])
def test_factors_below_the_normal_range(value, max_norm, dtype):
    """Factors that fp32 holds with a few bits only, or as 0."""
    import torch
    from sketch_attention_compression_b200 import clip_grad_norm
    gen = torch.Generator().manual_seed(3)
    g = [(torch.rand(n, generator=gen) * value).to(getattr(torch, dtype)).cuda() for n in (1001, 8, 300)]
    want64 = math.sqrt(math.fsum(float(x.double().square().sum()) for x in g))
    mul = max_norm / (want64 + 1e-6)
    assert mul < 2.0 ** -126
    out = [torch.zeros_like(x) for x in g]
    norm = clip_grad_norm(g, max_norm, out=out)
    assert abs(norm.item() - want64) <= 6 * E32 * want64
    for o, x in zip(out, g):
        w = x.double() * mul
        # fp32's (and bf16's) smallest spacings: 2^-149, 2^-133
        tol = (9 * E32 + (E16 if dtype == "bfloat16" else 0)) * w + \
            (2.0 ** -133 if dtype == "bfloat16" else 2.0 ** -149)
        assert ((o.double() - w).abs() <= tol).all()
    norm2 = clip_grad_norm(g, max_norm)
    assert torch.equal(norm, norm2) and all(torch.equal(a, b) for a, b in zip(g, out))
