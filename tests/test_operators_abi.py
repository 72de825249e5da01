"""The C entry points of linear attention, the block norms and the gradient
norm refuse bad host-side arguments before they touch the GPU (the addresses
here are no device memory; this runs without a GPU)."""

import ctypes
import os

import pytest

from sketch_attention_compression_b200 import binding

A = 1 << 20  # an aligned address nothing reads
BAD = binding.SA_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from sketch_attention_compression_b200 import build
        build.build()
    return binding.load_library()


def _forward(lib, **change):
    a = dict(q=A, qr=128, qh=64, k=A, kr=128, kh=64, v=A, vr=128, vh=64, g=A, off=A, batch=1,
             rows=10, longest=0, heads=2, dk=64, dv=64, dtype=0, scale=0.1, s0=None, out=A, fin=None,
             ws=A, n=1 << 30, st=None)
    assert set(change) <= set(a)
    return lib.sa_linear_attention_forward(*{**a, **change}.values())


def _backward(lib, **change):
    a = dict(q=A, qr=128, qh=64, k=A, kr=128, kh=64, v=A, vr=128, vh=64, g=A, off=A, batch=1,
             rows=10, longest=0, heads=2, dk=64, dv=64, dtype=0, scale=0.1, s0=None, do=A, dor=128,
             doh=64, ds=None, dq=A, dkk=A, dvv=A, ds0=None, ws=A, n=1 << 30, st=None)
    assert set(change) <= set(a)
    return lib.sa_linear_attention_backward(*{**a, **change}.values())


COMMON = [dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(off=None), dict(ws=None),
          dict(ws=A + 128), dict(off=A + 4), dict(q=A + 1), dict(batch=-1), dict(batch=1 << 21),
          dict(rows=-1), dict(rows=1 << 31), dict(longest=-1), dict(heads=0), dict(heads=1025),
          dict(dk=63), dict(dk=0), dict(dk=256), dict(dv=96), dict(dtype=2), dict(scale=0.0),
          dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e30), dict(qr=-1),
          dict(qh=63), dict(vh=0), dict(kr=1 << 41), dict(s0=A + 4), dict(batch=0)]


@pytest.mark.parametrize("change", COMMON + [dict(out=None), dict(out=A + 2), dict(fin=A + 8)])
def test_forward_refuses(lib, change):
    assert _forward(lib, **change) == BAD


@pytest.mark.parametrize("change", COMMON + [dict(do=None), dict(doh=10), dict(dq=None), dict(dkk=None),
                                             dict(dvv=A + 2), dict(ds=A + 4), dict(ds0=A + 4)])
def test_backward_refuses(lib, change):
    assert _backward(lib, **change) == BAD


def test_nothing_to_do(lib):
    assert _forward(lib, batch=0, rows=0, out=None) == binding.SA_OK
    assert lib.sa_workspace_bytes_linear_attention(0, 64, 64, 1, 1, 0) == 0
    assert lib.sa_workspace_bytes_linear_attention(1, 65, 64, 1, 1, 0) == 0
    assert lib.sa_workspace_bytes_grad_norm(-1) == 0


@pytest.mark.parametrize("change", [
    dict(q=None), dict(state=None), dict(out=None), dict(g=None), dict(batch=-1), dict(states=0),
    dict(heads=0), dict(dk=0), dict(dk=257), dict(dv=6), dict(dv=260), dict(dv=0), dict(dtype=5),
    dict(scale=float("nan")), dict(state=A + 4), dict(slots=A + 4), dict(qh=10), dict(flags=A + 2)])
def test_step_refuses(lib, change):
    a = dict(q=A, qr=128, qh=64, k=A, kr=128, kh=64, v=A, vr=128, vh=64, g=A, slots=None, batch=1,
             states=1, heads=2, dk=64, dv=64, dtype=0, scale=0.1, state=A, out=A, flags=None, st=None)
    assert lib.sa_linear_attention_step(*{**a, **change}.values()) == BAD
    assert lib.sa_linear_attention_step(*{**a, "batch": 0, "q": None}.values()) == binding.SA_OK


@pytest.mark.parametrize("change", [
    dict(x=None), dict(ldx=63), dict(ldy=63), dict(ldz=63), dict(x=A + 2), dict(y=A + 1), dict(d=0),
    dict(d=8193), dict(rows=-1), dict(rt=2), dict(rt=0, t=1), dict(kind=2), dict(gk=3), dict(eps=0.0),
    dict(eps=float("nan")), dict(r=None), dict(u=None), dict(g2=None), dict(g1=None), dict(y=None),
    dict(g1=A + 2)])
def test_block_norm_forward_refuses(lib, change):
    a = dict(x=A, ldx=64, y=A, ldy=64, z=A, ldz=64, g1=A, b1=A, rs=A, g2=A, b2=A, rows=3, d=64, rt=1,
             t=0, kind=0, gk=2, eps=1e-5, r=A, u=A, st=None)
    assert lib.sa_block_norm_forward(*{**a, **change}.values()) == BAD


@pytest.mark.parametrize("change", [
    dict(r=None), dict(dx=None), dict(dy=None), dict(dz=None), dict(du=None), dict(lddu=3),
    dict(lddr=3), dict(g1=None), dict(g2=None), dict(y=None), dict(eps=-1.0), dict(s1=A + 2)])
def test_block_norm_backward_refuses(lib, change):
    a = dict(r=A, ldr=64, y=A, ldy=64, z=A, ldz=64, g1=A, b1=A, rs=A, g2=A, rows=3, d=64, rt=1, t=0,
             kind=0, gk=2, eps=1e-5, dr=A, lddr=64, du=A, lddu=64, dx=A, dy=A, dz=A, s1=A, s2=A, s3=A,
             s4=A, s5=A, ws=A, n=1 << 30, st=None)
    assert lib.sa_block_norm_backward(*{**a, **change}.values()) == BAD


def _table(addresses, sizes, types):
    n = len(addresses)
    return ((ctypes.c_void_p * n)(*addresses), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int * n)(*types))


def test_clip_refuses(lib):
    ok = _table([A, A + 4096], [64, 64], [1, 0])
    tail = (A, 1 << 20, None)

    def clip(t=ok, out=None, n=2, max_norm=1.0, norm=A, tail=tail):
        return lib.sa_clip_grad_norm(t[0], out, t[1], t[2], n, max_norm, norm, *tail)

    for t in (_table([A, A], [64, 64], [1, 1]), _table([A, A + 100], [64, 64], [1, 1]),
              _table([A, A + 4096], [64, -1], [1, 1]), _table([A, None], [64, 4], [1, 1]),
              _table([A, A + 4096], [64, 64], [1, 2]), _table([A + 2, A + 4096], [64, 64], [1, 1])):
        assert clip(t) == BAD
    outs = (ctypes.c_void_p * 2)(A + 8, A + 8192)      # meets the first source
    assert clip(out=outs) == BAD
    assert clip(out=(ctypes.c_void_p * 2)(A + 8192, A + 8192)) == BAD
    assert clip(n=-1) == BAD and clip(norm=None) == BAD and clip(norm=A + 2) == BAD
    assert clip(tail=(None, 1 << 20, None)) == BAD and clip(tail=(A + 4, 1 << 20, None)) == BAD
    for max_norm in (-1.0, float("nan"), float("inf")):
        assert clip(max_norm=max_norm) == BAD
