"""Refusals of the norm and rotation and of cross attention, before anything is launched; no GPU needed."""
import ctypes

import pytest
import torch

from precision_attention_fa4fp4_gb300 import api, build

INVALID, UNSUP, ALIGN, WORK = 1, 2, 3, 6
vp, i, i64, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class Heads(ctypes.Structure):
    _fields_ = [("ptr", vp), ("b", i64), ("h", i64), ("n", i64)]


class Rotation(ctypes.Structure):
    _fields_ = [("positions", vp), ("shared", i), ("axes", i), ("sections", ctypes.POINTER(i)),
                ("freqs", ctypes.POINTER(ctypes.c_double)), ("interleaved", i)]


class Norm(ctypes.Structure):
    _fields_ = [("q_weight", vp), ("k_weight", vp), ("weight_dtype", i), ("eps", f)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load_library()


def heads(ptr=4096, b=64 * 64, h=64 * 8, n=64):
    return ctypes.byref(Heads(ptr, b, h, n))      # never dereferenced on the host


def rotation(axes=1, sections=(32,), freqs=None, positions=4096):
    s = (i * len(sections))(*sections)
    fr = (ctypes.c_double * 64)(*(freqs or [0.1] * 64))
    return ctypes.byref(Rotation(positions, 0, axes, s, fr, 0))


def norm(dtype=0, eps=1e-6, wq=None, wk=None):
    return ctypes.byref(Norm(wq, wk, dtype, eps))


def test_norm_rope_arguments(lib):
    call = lambda q=heads(), k=heads(), B=2, Hq=4, Hkv=2, N=8, d=64, n=norm(), r=rotation(), a=heads(), b=heads(): (
        lib.fa4fp4_norm_rope(q, k, B, Hq, Hkv, N, d, n, r, a, b, None))
    assert call(B=-1) == INVALID and call(N=-1) == INVALID
    assert call(d=96) == UNSUP and call(B=1 << 20, N=1 << 20) == UNSUP
    assert call(n=None, r=None) == INVALID
    assert call(k=None) == INVALID and call(q=None) == INVALID and call(b=None) == INVALID
    assert call(q=heads(ptr=None)) == INVALID
    assert call(q=heads(ptr=4097)) == ALIGN and call(a=heads(ptr=4104)) == ALIGN
    assert call(q=heads(n=60)) == ALIGN and call(k=heads(b=1028)) == ALIGN
    assert call(q=heads(n=-64)) == INVALID and call(q=heads(h=1 << 41)) == INVALID
    assert call(a=heads(h=0)) == INVALID          # rows of an output on each other
    assert call(n=norm(dtype=3)) == INVALID and call(n=norm(eps=-1.0)) == INVALID
    assert call(n=norm(eps=float("nan"))) == INVALID and call(n=norm(eps=float("inf"))) == INVALID
    assert call(n=norm(wq=4100)) == ALIGN
    assert call(r=rotation(axes=0)) == INVALID and call(r=rotation(axes=5, sections=(8,) * 5)) == INVALID
    assert call(r=rotation(sections=(31,))) == INVALID
    assert call(r=rotation(axes=2, sections=(33, -1))) == INVALID
    assert call(r=rotation(freqs=[float("nan")] * 64)) == INVALID
    assert call(r=rotation(positions=None)) == INVALID and call(r=rotation(positions=4098)) == ALIGN
    assert call(B=0, q=None, k=None, a=None, b=None, Hkv=0) == 0      # empty: nothing is looked at
    assert call(N=0, q=None, a=None, b=None) == 0


def test_norm_rope_bwd_arguments(lib):
    size = lib.fa4fp4_norm_rope_bwd_workspace_bytes
    assert size(0, 4, 2, 8, 64) == 0 and size(1, 4, 2, 0, 64) == 0 and size(1, 4, 2, 8, 96) == 0 and size(-1, 4, 2, 8, 64) == 0
    assert size(1, 4, 2, 8, 64) % 256 == 0 and size(1, 4, 2, 8, 64) >= 512
    call = lambda dy=heads(), t=0, n=norm(), r=rotation(), dq=heads(), dwq=4096, ws=4096, wn=1 << 30, d=64: (
        lib.fa4fp4_norm_rope_bwd(dy, heads(), t, heads(), heads(), 2, 4, 2, 8, d, n, r, dq, heads(), vp(dwq), vp(4096),
                                 vp(ws), sz(wn), None))
    assert call(t=2) == INVALID and call(dy=None) == INVALID and call(dq=heads(n=0)) == INVALID
    assert call(d=80) == UNSUP and call(n=None) == INVALID            # weight gradients without a norm
    assert call(ws=None) == WORK and call(wn=16) == WORK and call(ws=4100) == ALIGN
    assert call(dwq=4100) == ALIGN and call(dy=heads(n=62)) == ALIGN


def test_cross_arguments(lib):
    fwd = lambda q=heads(), k=heads(), v=heads(), lens=None, B=2, Hq=4, Hkv=2, Nq=8, Nk=8, d=64, o=heads(), lse=4096: (
        lib.fa4bf16_cross_fwd(q, k, v, vp(lens), B, Hq, Hkv, Nq, Nk, d, f(0.0), o, vp(lse), None))
    assert fwd(B=-1) == INVALID and fwd(Nk=-1) == INVALID
    assert fwd(d=32) == UNSUP and fwd(Hkv=3) == UNSUP and fwd(Hkv=0) == UNSUP and fwd(B=1 << 14, Nq=1 << 17) == UNSUP
    assert fwd(q=None) == INVALID and fwd(k=None) == INVALID and fwd(o=None) == INVALID
    assert fwd(o=heads(b=0)) == INVALID and fwd(v=heads(ptr=4100)) == ALIGN and fwd(k=heads(n=68)) == ALIGN
    assert fwd(lens=4098) == ALIGN and fwd(lse=4100) == ALIGN
    assert fwd(Nq=0, q=None, k=None, v=None, o=None) == 0
    size = lib.fa4bf16_cross_bwd_workspace_bytes
    assert size(0, 4, 2, 8, 8, 64) == 0 and size(1, 4, 3, 8, 8, 64) == 0
    assert size(2, 4, 2, 8, 8, 64) > 0 and size(2, 4, 2, 8, 8, 64) % 16 == 0
    bwd = lambda q=heads(), k=heads(), g=heads(), lse=4096, dq=heads(), dk=heads(), ws=4096, wn=1 << 30, d=64, Nq=8: (
        lib.fa4bf16_cross_bwd(q, k, heads(), heads(), g, vp(lse), None, 2, 4, 2, Nq, 8, d, f(0.0), dq, dk, heads(), vp(ws),
                              sz(wn), None))
    assert bwd(d=96) == UNSUP and bwd(q=None) == INVALID and bwd(g=None) == INVALID and bwd(lse=None) == INVALID
    assert bwd(dk=heads(n=0)) == INVALID and bwd(dq=heads(h=12)) == ALIGN
    assert bwd(ws=None) == WORK and bwd(wn=8) == WORK and bwd(ws=4104) == ALIGN


def test_python_refuses_what_it_can_see(lib):
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    for call in (lambda: api.qk_norm_rope(x, x), lambda: api.cross_fwd(x, x, x), lambda: api.cross_bwd(x, x, x, x, x, x),
                 lambda: api.qk_norm_rope_bwd(x, x, x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: api.qk_norm_rope(x[0], x), lambda: api.cross_fwd(x, x[0], x)):
        with pytest.raises(ValueError, match="dimensions"):
            call()
    with pytest.raises(TypeError):
        api.cross_fwd(x, x)
    with pytest.raises(TypeError):
        api.qk_norm_rope(x, x, positionz=1)


def test_rope_freqs():
    a = api.rope_freqs(128, (22, 21, 21), base=10000.0)
    assert a.dtype == torch.float64 and a.shape == (64,) and a[0] == a[22] == a[43] == 1
    assert abs(float(a[1]) - 10000.0 ** (-1 / 22)) < 1e-15 and abs(float(a[63]) - 10000.0 ** (-20 / 21)) < 1e-15
    assert torch.equal(api.rope_freqs(64), 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32))
    assert api.rope_freqs(64, (32, 0)).shape == (32,)
    for bad in (dict(d=64, sections=(30,)), dict(d=64, sections=(33, -1)), dict(d=63), dict(d=64, base=0.0)):
        with pytest.raises(ValueError):
            api.rope_freqs(**bad)
