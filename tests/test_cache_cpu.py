"""Host-side checks of the 8-bit cache's entry points that need no GPU: what
they refuse, empty problems, workspace sizes, and the reference's own pins."""
import ctypes
import struct

import numpy as np
import pytest
import torch

import cache_ref as R

OK, INVALID, UNSUP, ALIGN, WS = 0, 1, 2, 3, 6
P = ctypes.c_void_p(4096)           # never dereferenced: validation fails first
ODD = ctypes.c_void_p(4098)
BIG = 1 << 40


@pytest.fixture(scope="module")
def fa():
    from precision_attention_fa4fp4_gb300 import api, build
    build.build()
    api.load_library()
    return api


def cache(fa, ptrs=(4096,) * 5, n=8, H=2, page=64, d=128):
    """The C structure, as bytes."""
    return struct.pack("@5P4i", *(p or 0 for p in ptrs), n, H, page, d)


def calls(fa):
    """Every call with good arguments for B = 1, Hq = 4, T = 2, three pages;
    keyword arguments replace one."""
    lib = fa.load_library()
    cp, vp, i, f, sz = ctypes.c_char_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa4fp4_cache_append.argtypes = [cp] + [vp] * 5 + [i, i, i, vp]
    lib.fa4fp4_cache_fwd.argtypes = [cp] + [vp] * 5 + [i] * 5 + [f, i, vp, i, vp, vp, sz, vp]
    lib.fa4fp4_cache_select.argtypes = [cp] + [vp] * 4 + [i] * 5 + [vp, vp, sz, vp]
    lib.fa4fp4_cache_weigh.argtypes = [cp] + [vp] * 5 + [i] * 4 + [f, i, vp, vp, vp, sz, vp]
    lib.fa4fp4_cache_evict.argtypes = [cp] + [vp] * 4 + [i] * 5 + [vp] * 4

    def append(c, k=P, v=P, table=P, lens=P, n_new=None, B=1, mp=3, T=2):
        return lib.fa4fp4_cache_append(c, k, v, table, lens, n_new, B, mp, T, None)

    def fwd(c, q=P, table=P, lens=P, q_lens=None, pages=None, B=1, Hq=4, T=2, mp=3, n_sel=0, o=P, dt=1, lse=None,
            ws=P, wb=BIG):
        return lib.fa4fp4_cache_fwd(c, q, table, lens, q_lens, pages, B, Hq, T, mp, n_sel, 0.0, 1, o, dt, lse, ws, wb,
                                    None)

    def select(c, q=P, table=P, lens=P, q_lens=None, B=1, Hq=4, T=2, mp=3, n_sel=2, out=P, ws=P, wb=BIG):
        return lib.fa4fp4_cache_select(c, q, table, lens, q_lens, B, Hq, T, mp, n_sel, out, ws, wb, None)

    def weigh(c, q=P, lse=P, table=P, lens=P, q_lens=None, B=1, Hq=4, T=2, mp=3, w=P, out=P, ws=None,
              wb=0):
        return lib.fa4fp4_cache_weigh(c, q, lse, table, lens, q_lens, B, Hq, T, mp, 0.0, 1, w, out, ws, wb, None)

    def evict(c, table=P, lens=P, w=P, dst=P, B=1, mp=3, dp=2, budget=100, recent=4, nl=P, kept=P, wo=None):
        return lib.fa4fp4_cache_evict(c, table, lens, w, dst, B, mp, dp, budget, recent, nl, kept, wo, None)

    return dict(append=append, fwd=fwd, select=select, weigh=weigh, evict=evict)


@pytest.mark.parametrize("name", ["append", "fwd", "select", "weigh", "evict"])
def test_refusals(fa, name):
    f = calls(fa)[name]
    good = cache(fa)
    assert f(None) == INVALID
    assert f(cache(fa, d=96)) == UNSUP
    for page in (0, 8, 48, 256):
        assert f(cache(fa, page=page)) == UNSUP
    assert f(cache(fa, n=0)) == INVALID
    assert f(cache(fa, H=-1)) == INVALID
    assert f(good, mp=0) == INVALID
    assert f(good, mp=1 << 26) == UNSUP
    assert f(good, B=-1) == INVALID
    assert f(good, B=70000) == UNSUP
    for i in range(5):
        ptrs = [4096] * 5
        ptrs[i] = None
        assert f(cache(fa, ptrs)) == INVALID
        ptrs[i] = 4098
        assert f(cache(fa, ptrs)) == ALIGN
    assert f(good, table=None) == INVALID
    assert f(good, lens=None) == INVALID
    assert f(good, lens=ODD) == ALIGN
    assert f(good, table=ODD) == ALIGN
    # an empty batch is a no-op that looks at no pointer but the structure
    assert f(cache(fa, (None,) * 5), B=0, table=None, lens=None) == OK
    assert f(cache(fa, (None,) * 5, page=48), B=0) == UNSUP


def test_refusals_of_each_call(fa):
    c, good = calls(fa), cache(fa)
    odd4 = ctypes.c_void_p(4100)
    assert c["append"](good, k=None) == INVALID
    assert c["append"](good, v=odd4) == ALIGN
    assert c["append"](good, T=-1) == INVALID
    assert c["append"](good, T=0, k=None, v=None) == OK
    assert c["fwd"](good, q=None) == INVALID
    assert c["fwd"](good, o=None) == INVALID
    assert c["fwd"](good, dt=2) == INVALID
    assert c["fwd"](good, Hq=5) == UNSUP
    assert c["fwd"](good, q=odd4) == ALIGN
    assert c["fwd"](good, lse=odd4) == ALIGN
    assert c["fwd"](good, n_sel=3) == INVALID             # a count without a list
    assert c["fwd"](good, pages=P, n_sel=0) == INVALID    # a list without a count
    assert c["fwd"](good, ws=None) == WS
    need = fa.load_library().fa4fp4_cache_fwd_workspace_bytes(1, 4, 2, 2, 128, 64, 3, 0)
    assert c["fwd"](good, wb=need - 1) == WS
    assert c["fwd"](good, ws=odd4, wb=need) == ALIGN
    assert c["fwd"](good, T=1 << 30, Hq=4) == UNSUP
    assert c["fwd"](cache(fa, H=64), B=65535, Hq=64, T=1, mp=1 << 20) == UNSUP     # 2^31 units or more
    assert c["fwd"](cache(fa, n=1 << 24, H=8), Hq=8) == UNSUP                      # 2^31 pool rows or more
    assert c["fwd"](good, T=0, q=None, o=None, ws=None) == OK
    assert c["select"](good, n_sel=0) == INVALID
    assert c["select"](good, out=None) == INVALID
    assert c["select"](good, mp=16385, wb=1 * 2 * 2 * 16385 * 8 - 1) == WS
    assert c["select"](good, mp=16385, ws=None) == WS
    assert c["select"](good, mp=16385, ws=odd4) == ALIGN
    assert c["select"](cache(fa, page=16), mp=(1 << 18) + 1) == UNSUP
    assert c["weigh"](good, lse=None) == INVALID
    assert c["weigh"](good, w=None) == INVALID
    assert c["weigh"](good, out=ODD) == ALIGN
    need = fa.cache_weigh_workspace_bytes(1, 4, 2, 64, 128)
    assert c["weigh"](good, T=64) == WS and c["weigh"](good, T=64, ws=P, wb=need - 1) == WS
    assert c["weigh"](good, T=64, ws=odd4, wb=need) == ALIGN
    assert c["evict"](good, budget=0) == INVALID
    assert c["evict"](good, budget=129) == INVALID        # more than two pages of 64 hold
    assert c["evict"](good, recent=101) == INVALID
    assert c["evict"](good, recent=-1) == INVALID
    assert c["evict"](good, dp=0) == INVALID
    assert c["evict"](good, kept=None) == INVALID
    assert c["evict"](good, wo=ODD) == ALIGN


def test_workspace_sizes(fa):
    f = fa.cache_fwd_workspace_bytes
    # one unit per kv head: a counter word and two slots of eight rows (d
    # values, max and sum) each
    assert f(1, 8, 2, 1, 128, 64, 2, 0) == 2 * 8 + 2 * 2 * 8 * 130 * 4
    assert f(1, 8, 2, 1, 128, 64, 0, 0) == 0 and f(1, 8, 3, 1, 128, 64, 2, 0) == 0
    assert f(0, 8, 2, 1, 128, 64, 2, 0) == 0
    assert f(65535, 64, 64, 1, 128, 128, 1 << 20, 0) == 0 and f(1, 8, 2, 1, 128, 64, 2, 1 << 25) == 0
    # bounded by the grid, whatever the batch
    assert f(512, 64, 8, 1, 128, 64, 4096, 0) == f(64, 64, 8, 1, 128, 64, 4096, 0) < (8 << 20)
    # tiles of 128 rows of f16 and 16 bytes of constants a row, from 80 rows on
    assert fa.cache_weigh_workspace_bytes(1, 4, 2, 31, 128) == 0
    assert fa.cache_weigh_workspace_bytes(3, 4, 2, 65, 64) == 3 * 2 * 2 * 128 * (64 * 2 + 16)
    assert fa.cache_select_workspace_bytes(2, 3, 4, 16384) == 0
    assert fa.cache_select_workspace_bytes(2, 3, 4, 16385) == 2 * 3 * 4 * 16385 * 8


def test_binding_refuses_cpu_tensors(fa):
    z = torch.zeros((4, 2, 64, 128), dtype=torch.uint8)
    with pytest.raises(ValueError):
        fa.KVCache(z, z, z[:, :, 0, 0].contiguous(), z[:, :, 0, 0].contiguous(), z[:, :, :2].contiguous())
    with pytest.raises(ValueError):
        fa.KVCache(z[0], z, z, z, z)
    with pytest.raises(ValueError):
        fa.KVCache(*[None] * 5)
    t = torch.zeros((1, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.cache_append(None, z, z, t, t[:, 0])
    for args, kw in (((), {}), ((None,) * 7, {}), ((None,) * 5, dict(lens=t)), ((None,) * 5, dict(tokens=t))):
        with pytest.raises(TypeError):
            fa.cache_append(*args, **kw)
    with pytest.raises(TypeError):
        fa.KVCache(z)


def test_status_strings(fa):
    lib = fa.load_library()
    assert b"range" in lib.fa4fp4_status_string(7)
    assert b"infinity" in lib.fa4fp4_status_string(8)
    assert lib.fa4fp4_status_string(9) == b"unknown status"


def test_reference_rounding():
    """The reference's E4M3 codes against torch's conversion, its exponents
    against the definition."""
    x = torch.cat([torch.linspace(-460, 460, 20001), torch.logspace(-12, 2.5, 5001), torch.tensor([0.0, -0.0])])
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.e4m3_codes(x.double().numpy()), want)
    for a in (0.0, 1e-45, 447.9, 448.0, 448.1, 512.0, 895.9, 896.0, 897.0, 3e38):
        X = R.least_exponent(a)
        assert a <= 448 * 2.0 ** X and (X == -127 or a > 448 * 2.0 ** (X - 1))
