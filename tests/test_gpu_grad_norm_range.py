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
