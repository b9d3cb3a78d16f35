"""Cross attention, forward and backward, against plain forms in 64 bits."""
import pytest
import torch

import layer_ref as ref
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def fa():
    return require_gpu()


def make(B, Hq, Hkv, Nq, Nk, d, lens=None, seed=0, size=1.0):
    """q dense, k and v views of one projection; `lens` a list, behind which k and v hold NaN and infinities."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (torch.randn((B, Hq, Nq, d), generator=g, device="cuda") * size).to(torch.bfloat16)
    kv = torch.randn((B, Nk, 2, Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    if lens is not None:
        for b, n in enumerate(lens):
            kv[b, n:] = float("nan")
            kv[b, n + 1:: 3] = INF
        lens = torch.tensor(lens, device="cuda", dtype=torch.int32)
    return q, kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2), lens, g


def check_fwd(fa, q, k, v, lens, scale=0.0, **more):
    o, lse = fa.cross_fwd(q, k, v, lens, softmax_scale=scale, **more)
    fa.sync_status()
    want, bo, wl, bl = ref.cross(q, k, v, lens, scale)
    ref.assert_within(o, want, bo, "o")
    dead = wl == -INF
    assert torch.equal(lse == -INF, dead)
    ref.assert_within(lse.masked_fill(dead, 0), wl.masked_fill(dead, 0), bl, "lse")
    return o, lse


def check_bwd(fa, q, k, v, lens, g, scale=0.0, **more):
    o, lse = fa.cross_fwd(q, k, v, lens, softmax_scale=scale)
    dout = torch.randn(q.shape, generator=g, device="cuda").to(torch.bfloat16)
    got = fa.cross_bwd(q, k, v, o, dout, lse, lens, softmax_scale=scale, **more)
    fa.sync_status()
    for name, x, (want, bound) in zip(("dq", "dk", "dv"), got, ref.cross_bwd(q, k, v, o, dout, lse, lens, scale)):
        ref.assert_within(x, want, bound, name)
    again = fa.cross_bwd(q, k, v, o, dout, lse, lens, softmax_scale=scale)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    return got


# (B, Hq, Hkv, Nq, Nk, lens)
SHAPES = [
    (1, 1, 1, 1, 1, None), (2, 4, 4, 1, 0, None), (2, 4, 2, 3, 7, [7, 0]), (3, 8, 1, 1, 300, [1, 300, 33]),
    (2, 6, 2, 5, 1000, [999, 513]), (1, 16, 2, 2, 64, None), (1, 7, 1, 1, 129, None), (4, 2, 2, 16, 31, [31, 30, 16, 1]),
    (1, 2, 2, 17, 128, None), (2, 3, 3, 100, 77, [77, 20]), (1, 4, 1, 33, 257, None), (1, 2, 1, 127, 256, None),
    (2, 2, 2, 128, 129, [128, 129]), (1, 2, 2, 129, 512, None), (2, 2, 1, 256, 200, [0, 130]), (1, 1, 1, 257, 700, None),
    (1, 4, 2, 300, 127, [100]), (3, 1, 1, 513, 384, [384, 256, 255]), (1, 2, 2, 1000, 1, None), (2, 2, 2, 40, 2000, [1999, 3]),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk,lens", SHAPES)
def test_forward(fa, d, B, Hq, Hkv, Nq, Nk, lens):
    check_fwd(fa, *make(B, Hq, Hkv, Nq, Nk, d, lens)[:4])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk,lens", SHAPES)
def test_backward(fa, d, B, Hq, Hkv, Nq, Nk, lens):
    check_bwd(fa, *make(B, Hq, Hkv, Nq, Nk, d, lens))


# shapes where the work of one head is spread over the GPU: clusters of every size, row groups, query tiles and key
# tiles whose steps lie in several ranges
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk,lens", [
    (1, 1, 1, 1, 4100, None), (1, 8, 1, 2, 16000, None), (1, 6, 2, 33, 2500, None), (2, 1, 1, 40, 5000, [4999, 17]),
    (1, 1, 1, 100, 3001, None), (1, 1, 1, 256, 9000, [8999]), (5, 3, 3, 9, 1100, [1100, 0, 1, 513, 512]),
    (1, 1, 1, 13, 6000, None), (1, 2, 1, 1500, 257, [129]), (3, 2, 1, 700, 900, [900, 300, 601])])
def test_spread(fa, d, B, Hq, Hkv, Nq, Nk, lens):
    q, k, v, lens, g = make(B, Hq, Hkv, Nq, Nk, d, lens)
    check_fwd(fa, q, k, v, lens)
    check_bwd(fa, q, k, v, lens, g)


@pytest.mark.parametrize("d", [64, 128])
def test_fewer_steps_than_room(fa, d):
    """Most sequences are empty: there are more multiprocessors than steps, and ranges without any."""
    for lens in ([0] * 39 + [130], [0] * 40, [1] + [0] * 38 + [600]):
        q, k, v, lens, g = make(40, 4, 2, 300, 600, d, lens)
        check_fwd(fa, q, k, v, lens)
        dq, dk, dv = check_bwd(fa, q, k, v, lens, g)
        assert (dk[1:39] == 0).all() and (dv[1:39] == 0).all() and (dq[1:39] == 0).all()


def test_one_key(fa):
    """One key: o is its value, and dQ and dK are zero but for roundings of P = 1 (dS = dP - D)."""
    q, k, v, _, g = make(2, 2, 2, 150, 1, 64)
    o, lse = check_fwd(fa, q, k, v, None)
    assert torch.equal(o, v.expand(-1, -1, 150, -1))
    check_bwd(fa, q, k, v, None, g)


def test_refusals(fa):
    q, k, v, _, _ = make(1, 2, 2, 4, 8, 64)
    c = k.contiguous()
    with pytest.raises(fa.api.Fa4Fp4Error):
        fa.cross_fwd(q, c.as_strided((1, 2, 8, 64), (1024, 512, 32, 1)), v)        # rows on each other
    with pytest.raises(fa.api.Fa4Fp4Error):
        fa.cross_fwd(q, k, v, out=q.new_empty((1, 1, 4, 64)).expand(-1, 2, -1, -1))   # outputs on each other
    for bad in (dict(kv_lens=torch.zeros(2, device="cuda", dtype=torch.int32)), dict(kv_lens=torch.zeros(1, device="cuda")),
                dict(out=q.float()), dict(lse=q)):
        with pytest.raises(ValueError):
            fa.cross_fwd(q, k, v, **bad)
    with pytest.raises(ValueError):
        fa.cross_fwd(q, k, v[:, :1])
    with pytest.raises(ValueError):
        fa.cross_fwd(q, k.transpose(2, 3).contiguous().transpose(2, 3), v)
    o, lse = fa.cross_fwd(q, k, v)
    with pytest.raises(fa.api.Fa4Fp4Error):
        fa.cross_bwd(q, k, v, o, q, lse, workspace=torch.empty(16, device="cuda", dtype=torch.uint8))
    w = torch.empty(fa.cross_bwd_workspace_bytes(1, 2, 2, 4, 8, 64), device="cuda", dtype=torch.uint8)
    for a, b in zip(fa.cross_bwd(q, k, v, o, q, lse, workspace=w), fa.cross_bwd(q, k, v, o, q, lse)):
        assert torch.equal(a, b)
    fa.sync_status()


@pytest.mark.parametrize("Nq", [1, 4, 200])
def test_scores_of_every_size(fa, Nq):
    """Peaked, flat and negative rows; the largest score in the first, last and a middle key."""
    for d, size, scale in ((128, 30.0, 0.0), (64, 1e-4, 0.0), (128, 1.0, 4.0), (64, 1.0, 1e-6)):
        q, k, v, _, g = make(1, 4, 2, Nq, 333, d, size=size)
        check_fwd(fa, q, k, v, None, scale)
        check_bwd(fa, q, k, v, None, g, scale)
    q, k, v, _, _ = make(1, 1, 1, Nq, 640, 64)
    for at in (0, 639, 300):
        kk = k.clone()
        kk[0, 0, at] = q[0, 0, 0] * 40
        check_fwd(fa, q, kk, v, None)
    kk = k.clone()
    kk[:] = -q[0, 0, 0] * 20          # all scores of the first row far below zero, and equal
    check_fwd(fa, q, kk, v, None)


def test_rising_scores(fa):
    """Every block of keys raises the running maximum, by little and by much."""
    for step in (0.05, 3.0, 60.0):
        q, k, v, _, g = make(1, 2, 2, 150, 900, 64)
        q[...] = 1.0
        ramp = (torch.arange(900, device="cuda") // 64 * step / 8).to(torch.bfloat16)
        k = (k * 0.1 + ramp[:, None]).contiguous()
        check_fwd(fa, q, k, v, None)
        check_fwd(fa, q, k.flip(2), v, None)
        check_bwd(fa, q, k, v, None, g)


def test_large_and_zero_values(fa):
    """V that falls and rises by many binades, runs of zeros."""
    q, k, v, _, g = make(2, 2, 2, 140, 520, 128)
    v = v.clone()
    v[0, :, 100:300] = 0
    v[0, :, 300:] *= 2.0 ** 60
    v[1, :, :200] *= 2.0 ** 80
    v[1, :, 200:] *= 2.0 ** -60
    check_fwd(fa, q, k, v, None)
    check_fwd(fa, q[:, :, :3], k, v, None)


@pytest.mark.parametrize("Nq", [2, 200])
def test_strides_and_outputs(fa, Nq):
    """Queries in [B, N, H, d], outputs into views of it, broadcast keys; what lies between stays."""
    q, k, v, _, g = make(2, 4, 4, Nq, 150, 64)
    want, lse = check_fwd(fa, q, k, v, None)
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)
    room = torch.full((2, Nq, 6, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    out = room[:, :, 1:5].transpose(1, 2)
    l = torch.zeros_like(lse)
    o, l2 = fa.cross_fwd(qt, k.contiguous(), v.contiguous(), out=out, lse=l)
    assert o is out and l2 is l and torch.equal(out, want) and torch.equal(l, lse)
    assert (room[:, :, 0] == 7).all() and (room[:, :, 5] == 7).all()
    assert fa.cross_fwd(qt, k, v, with_lse=False)[1] is None
    kb, vb = k[:1].expand(2, -1, -1, -1), v[:, :1].expand(-1, 4, -1, -1)
    check_fwd(fa, q, kb, vb, None)
    check_bwd(fa, q, kb, vb, None, g)
    grads = [torch.full((2, n, 6, 64), 7.0, device="cuda", dtype=torch.bfloat16) for n in (Nq, 150, 150)]
    views = [x[:, :, 1:5].transpose(1, 2) for x in grads]
    dout = torch.randn(q.shape, generator=g, device="cuda").to(torch.bfloat16)
    plain = fa.cross_bwd(q, k, v, want, dout, lse)
    got = fa.cross_bwd(qt, k, v, want, dout, lse, dq=views[0], dk=views[1], dv=views[2])
    for a, b, room in zip(plain, got, grads):
        assert torch.equal(a, b) and (room[:, :, 0] == 7).all() and (room[:, :, 5] == 7).all()


def test_odd_base_and_row_strides(fa):
    """Views whose rows start at any multiple of 16 bytes."""
    g = torch.Generator(device="cuda").manual_seed(5)
    big = torch.randn((2, 300, 4 * 72), generator=g, device="cuda").to(torch.bfloat16)
    k = big[:, 3:, 8:264].unflatten(-1, (4, 64)).transpose(1, 2)
    v = big[:, 2:299, 16:272].unflatten(-1, (4, 64)).transpose(1, 2)
    q = big[:, :131, 24:280].unflatten(-1, (4, 64)).transpose(1, 2)
    check_fwd(fa, q, k, v, torch.tensor([297, 111], device="cuda", dtype=torch.int32))
    check_fwd(fa, q[:, :, 5:7], k, v, None)
    check_bwd(fa, q, k, v, torch.tensor([297, 111], device="cuda", dtype=torch.int32), g)


def test_far_offsets(fa):
    """Element offsets that pass 32 bits."""
    room = torch.empty(2 ** 31 + 2 ** 20, device="cuda", dtype=torch.bfloat16)
    k, v = (room[at:].as_strided((2, 2, 100, 64), (2 ** 31, 6400, 64, 1)) for at in (0, 2 ** 16))
    q, k0, v0, _, g = make(2, 2, 2, 150, 100, 64)
    k.copy_(k0)
    v.copy_(v0)
    for rows in (q, q[:, :, :2]):
        assert torch.equal(fa.cross_fwd(rows, k, v)[0], fa.cross_fwd(rows, k0, v0)[0])
    check_bwd(fa, q, k, v, None, g)


def test_length_out_of_range(fa):
    q, k, v, _, g = make(3, 2, 2, 4, 50, 64)
    for rows in (q, torch.cat([q] * 40, 2)):
        lens = torch.tensor([-1, 51, 20], device="cuda", dtype=torch.int32)
        o, lse = fa.cross_fwd(rows, k, v, lens)
        with pytest.raises(fa.api.Fa4Fp4Error) as e:
            fa.sync_status()
        assert e.value.status == 7
        fa.sync_status()
        a, b = fa.cross_fwd(rows, k, v, lens.clamp(0, 50))
        assert torch.equal(o, a) and torch.equal(lse, b) and (lse[0] == -INF).all()


def test_many_heads_and_sequences(fa):
    check_fwd(fa, *make(300, 12, 12, 1, 20, 64)[:4])
    q, k, v, lens, g = make(70, 8, 4, 20, 30, 64, [i % 31 for i in range(70)])
    check_fwd(fa, q, k, v, lens)
    check_bwd(fa, q, k, v, lens, g)


def test_two_calls_at_once(fa):
    """Two streams, each with a workspace of its own."""
    q, k, v, lens, g = make(2, 8, 4, 500, 700, 128, [700, 200])
    o, lse = fa.cross_fwd(q, k, v, lens)
    dout = torch.randn(q.shape, generator=g, device="cuda").to(torch.bfloat16)
    want = fa.cross_bwd(q, k, v, o, dout, lse, lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                a, b = fa.cross_fwd(q, k, v, lens)
                got[i] = (a, b, *fa.cross_bwd(q, k, v, a, dout, b, lens))
    torch.cuda.synchronize()
    for x in got:
        assert all(torch.equal(a, b) for a, b in zip(x, (o, lse, *want)))


@pytest.mark.parametrize("Nq", [1, 300])
def test_graph(fa, Nq):
    """A captured forward and backward, replayed on new inputs and lengths."""
    q, k, v, _, g = make(2, 4, 2, Nq, 400, 64)
    lens = torch.tensor([400, 399], device="cuda", dtype=torch.int32)
    dout = torch.randn(q.shape, generator=g, device="cuda").to(torch.bfloat16)
    fa.cross_bwd(q, k, v, *(lambda o, l: (o, dout, l))(*fa.cross_fwd(q, k, v, lens)), lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o, lse = fa.cross_fwd(q, k, v, lens)
        grads = fa.cross_bwd(q, k, v, o, dout, lse, lens)
    torch.cuda.synchronize()
    q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
    lens.copy_(torch.tensor([17, 0]))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    o2, lse2 = check_fwd(fa, q, k, v, lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for a, b in zip(grads, fa.cross_bwd(q, k, v, o2, dout, lse2, lens)):
        assert torch.equal(a, b)


def test_nothing_to_attend(fa):
    q, k, v, _, g = make(2, 4, 2, 6, 0, 64)
    dq, dk, dv = check_bwd(fa, q, k, v, None, g)
    assert (dq == 0).all() and dk.shape == (2, 2, 0, 64)
    q, k, v, _, g = make(2, 4, 2, 0, 9, 64)
    o, lse = fa.cross_fwd(q, k, v)
    assert o.shape == (2, 4, 0, 64)
    dq, dk, dv = fa.cross_bwd(q, k, v, o, q, lse)
    assert (dk == 0).all() and (dv == 0).all()
    e = torch.zeros((0, 4, 5, 64), device="cuda", dtype=torch.bfloat16)
    assert fa.cross_fwd(e, e, e)[0].shape == e.shape
    fa.sync_status()


def test_gradients_against_differences():
    """The plain form's own gradients, by central differences."""
    g = torch.Generator().manual_seed(1)
    q, k, v, dout = (torch.randn(s, generator=g, dtype=torch.float64) for s in
                     ((1, 2, 3, 64), (1, 1, 5, 64), (1, 1, 5, 64), (1, 2, 3, 64)))
    lens = torch.tensor([4])
    o, _, lse, _ = ref.cross(q, k, v, lens)
    grads = ref.cross_bwd(q, k, v, o, dout, lse, lens)
    for i, x in enumerate((q, k, v)):
        for at in ((0, 0, 1, 5), (0, x.shape[1] - 1, 2, 60)):
            was = float(x[at])
            f = []
            for e in (1e-5, -1e-5):
                x[at] = was + e
                f.append(float((ref.cross(q, k, v, lens)[0] * dout).sum()))
            x[at] = was
            assert abs((f[0] - f[1]) / 2e-5 - float(grads[i][0][at])) < 1e-7


@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk", [
    (1, 3, 3, 2500, 256), (2, 4, 2, 1200, 300), (1, 5, 5, 900, 512), (3, 2, 1, 700, 640), (1, 7, 7, 300, 768),
    (2, 6, 3, 520, 1000), (1, 1, 1, 3000, 1900), (5, 8, 2, 20, 257)])
def test_key_tiles_side_by_side(fa, B, Hq, Hkv, Nq, Nk):
    """Two to eight key tiles of a head go through its queries at the same time, and their ranges end inside lines;
    with lengths (all keys) each goes by itself."""
    q, k, v, _, g = make(B, Hq, Hkv, Nq, Nk, 128)
    check_bwd(fa, q, k, v, None, g)
    check_bwd(fa, q, k, v, torch.full((B,), Nk, device="cuda", dtype=torch.int32), g)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk,lens", [
    (1, 2, 1, 9000, 200, None), (1, 1, 1, 20000, 40, [39]), (1, 4, 1, 20, 16000, None), (2, 1, 1, 7, 9000, [9000, 1])])
def test_many_ranges_of_a_tile(fa, d, B, Hq, Hkv, Nq, Nk, lens):
    """One or two output tiles, whose sums come from most of the GPU."""
    q, k, v, lens, g = make(B, Hq, Hkv, Nq, Nk, d, lens)
    check_bwd(fa, q, k, v, lens, g)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk,lens", [
    (1, 7, 1, 241, 1590, [1234]), (3, 2, 1, 5985, 87, None), (7, 4, 1, 500, 66, [66, 1, 0, 65, 20, 0, 3]),
    (40, 2, 2, 130, 129, None), (40, 2, 2, 130, 129, [129, 0, 128, 5] * 10), (9, 7, 1, 33, 271, None)])
def test_joins(fa, d, B, Hq, Hkv, Nq, Nk, lens):
    """Output tiles of a few ranges and of many, fewer of them than ranges and more, sequences without keys between."""
    q, k, v, lens, g = make(B, Hq, Hkv, Nq, Nk, d, lens)
    check_bwd(fa, q, k, v, lens, g)
