"""Norm and rotation of queries and keys against plain forms in 64 bits."""
import pytest
import torch

import layer_ref as ref
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

SECTIONS = {1: lambda h: [h], 2: lambda h: [h // 2, h - h // 2], 3: lambda h: [h - 2 * (h // 3), h // 3, h // 3],
            4: lambda h: [h - 5, 0, 5, 0]}


@pytest.fixture(scope="module")
def fa():
    return require_gpu()


def make(B, Hq, Hkv, N, d, axes=1, far=1000, seed=0, fused=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((B, N, Hq + 2 * Hkv, d), generator=g, device="cuda") * 2).to(torch.bfloat16)
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq: Hq + Hkv].transpose(1, 2)
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    w = [1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]
    pos = torch.randint(-far, far + 1, (B, axes, N), generator=g, device="cuda").int()
    return q, k, w, pos, g


def both(fa, q, k, w, pos, freqs, sections, interleaved, norm=True, eps=1e-6, **more):
    ws = dict(q_weight=w[0], k_weight=w[1]) if w else {}
    out = fa.qk_norm_rope(q, k, pos, freqs, sections=sections, interleaved=interleaved, norm=norm, eps=eps, **ws, **more)
    if pos is not None and pos.dim() == 2:
        pos = pos[None].expand(q.shape[0], -1, -1)
    th = None if pos is None else ref.turns(pos, freqs, sections or [q.shape[-1] // 2])
    for name, y, x, wx in zip("qk", out, (q, k), w or (None, None)):
        if x is not None:
            ref.assert_within(y, *ref.norm_rope(x, wx, th, interleaved, norm, eps), name)
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,N,axes", [(1, 1, 1, 1, 1), (3, 5, 2, 1, 1), (2, 8, 8, 7, 2), (1, 3, 1, 33, 3),
                                             (2, 24, 24, 129, 3), (1, 32, 8, 300, 4), (64, 32, 8, 1, 1), (5, 7, 0, 17, 1)])
def test_forward(fa, d, interleaved, B, Hq, Hkv, N, axes):
    q, k, w, pos, _ = make(B, Hq, max(Hkv, 1), N, d, axes)
    sections = SECTIONS[axes](d // 2)
    freqs = fa.rope_freqs(d, sections)
    if Hkv == 0:
        out = fa.qk_norm_rope(q, None, pos, freqs, w[0], sections=sections, interleaved=interleaved)
        assert out[1] is None
        th = ref.turns(pos, freqs, sections)
        ref.assert_within(out[0], *ref.norm_rope(q, w[0], th, interleaved, True, 1e-6), "q")
    else:
        both(fa, q, k, w, pos, freqs, sections, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_forward_parts(fa, interleaved):
    """Norm alone, rotation alone, no weights, bf16 weights, shared positions, eps, other frequencies."""
    q, k, w, pos, g = make(2, 6, 3, 45, 64, 1, far=70000)
    freqs = fa.rope_freqs(64, base=500000.0)
    both(fa, q, k, w, None, None, None, interleaved)
    both(fa, q, k, None, pos, freqs, None, interleaved, norm=False)
    both(fa, q, k, None, pos, freqs, None, interleaved, eps=0.5)
    both(fa, q, k, [x.to(torch.bfloat16) for x in w], pos[0], freqs, None, interleaved)
    both(fa, q, k, w, pos, torch.linspace(-6.28, 6.28, 32, dtype=torch.float64), None, interleaved)
    some = freqs.clone()
    some[8:] = 0.0                      # the rest of the channels stays where it is
    both(fa, q, k, w, pos, some, None, interleaved)


def test_far_positions(fa):
    """Angles of positions up to the end of int32 are as exact as those near 0."""
    q, k, w, _, g = make(2, 4, 2, 64, 128)
    for far in (10 ** 6, 2 ** 31 - 1):
        pos = torch.randint(-far, far, (2, 1, 64), generator=g, device="cuda").int()
        pos[0, 0, 0], pos[1, 0, 0] = far, -far
        both(fa, q, k, w, pos, fa.rope_freqs(128), None, False)


def test_zero_and_large_rows(fa):
    q, k, w, pos, _ = make(1, 4, 4, 8, 128, fused=False)
    q[0, 0] = 0.0
    k[0, 1] *= 2.0 ** 50
    q[0, 2] *= 2.0 ** -40
    both(fa, q, k, w, pos, fa.rope_freqs(128), None, True)
    y, _ = fa.qk_norm_rope(q, k, pos, fa.rope_freqs(128), eps=1e-6)
    assert (y[0, 0] == 0).all()


def test_outputs_strided_and_in_place(fa):
    q, k, w, pos, _ = make(2, 4, 2, 19, 128)
    freqs = fa.rope_freqs(128)
    want = both(fa, q, k, w, pos, freqs, None, False)
    room = torch.full((2, 19, 9, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    out = room[:, :, :4].transpose(1, 2), room[:, :, 5:7].transpose(1, 2)
    got = fa.qk_norm_rope(q, k, pos, freqs, *w, q_out=out[0], k_out=out[1])
    assert got[0] is out[0] and got[1] is out[1]
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert (room[:, :, 4] == 7).all() and (room[:, :, 7:] == 7).all()
    fa.qk_norm_rope(q, k, pos, freqs, *w, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_broadcast_input(fa):
    q, k, w, pos, _ = make(1, 4, 2, 19, 128)
    q3 = q.expand(3, -1, -1, -1)
    kh = k[:, :1].expand(3, 5, -1, -1)
    both(fa, q3, kh, w, pos.expand(3, -1, -1).contiguous(), fa.rope_freqs(128), None, False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,N,axes,interleaved", [(1, 1, 1, 1, 1, True), (3, 5, 2, 1, 1, False),
                                                         (2, 8, 8, 7, 2, True), (1, 3, 1, 333, 3, False),
                                                         (2, 24, 24, 129, 3, True), (1, 32, 8, 2000, 1, False)])
def test_backward(fa, d, f32, B, Hq, Hkv, N, axes, interleaved):
    q, k, w, pos, g = make(B, Hq, Hkv, N, d, axes)
    sections = SECTIONS[axes](d // 2)
    freqs = fa.rope_freqs(d, sections)
    dy = [torch.randn(x.shape, generator=g, device="cuda").to(torch.float32 if f32 else torch.bfloat16) for x in (q, k)]
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(*dy, q, k, pos, freqs, *w, sections=sections, interleaved=interleaved)
    th = ref.turns(pos, freqs, sections)
    for name, got, gotw, x, y, wx in (("q", dq, dwq, q, dy[0], w[0]), ("k", dk, dwk, k, dy[1], w[1])):
        dx, bx, dw, bw = ref.norm_rope_bwd(y, x, wx, th, interleaved, True, 1e-6)
        ref.assert_within(got, dx, bx, "d" + name)
        ref.assert_within(gotw, dw, bw, f"d{name}_weight")
    again = fa.qk_norm_rope_bwd(*dy, q, k, pos, freqs, *w, sections=sections, interleaved=interleaved)
    assert all(torch.equal(a, b) for a, b in zip(again, (dq, dk, dwq, dwk)))


def test_backward_parts(fa):
    q, k, w, pos, g = make(2, 4, 2, 30, 64)
    freqs = fa.rope_freqs(64)
    th = ref.turns(pos, freqs, [32])
    dyq = torch.randn((2, 30, 4, 64), generator=g, device="cuda").transpose(1, 2)      # strided f32
    dyk = torch.randn((2, 30, 2, 64), generator=g, device="cuda").transpose(1, 2)
    # the rotation alone
    dq, dk, a, b = fa.qk_norm_rope_bwd(dyq, dyk, q, k, pos, freqs, norm=False)
    assert a is None and b is None
    ref.assert_within(dk, *ref.norm_rope_bwd(dyk, k, None, th, False, False, 0)[:2], "dk")
    # the norm alone, queries alone, one weight, into a slice of a fused gradient
    room = torch.zeros((2, 30, 8, 64), device="cuda", dtype=torch.bfloat16)
    at = room[:, :, :4].transpose(1, 2)
    dq, dk, a, b = fa.qk_norm_rope_bwd(dyq, None, q, None, q_weight=w[0], dq=at)
    assert dq is at and dk is None and b is None
    dx, bx, dw, bw = ref.norm_rope_bwd(dyq, q, w[0], None, False, True, 1e-6)
    ref.assert_within(dq, dx, bx, "dq")
    ref.assert_within(a, dw, bw, "dq_weight")
    assert (room[:, :, 4:] == 0).all()
    # no weights
    dq, dk, a, b = fa.qk_norm_rope_bwd(dyq, dyk, q, k, pos, freqs)
    assert a is None and b is None
    ref.assert_within(dq, *ref.norm_rope_bwd(dyq, q, None, th, False, True, 1e-6)[:2], "dq")


def test_backward_against_differences(fa):
    """The formula of the plain form itself, by central differences."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(1, 1, 2, 64, generator=g, dtype=torch.float64)
    dy = torch.randn(1, 1, 2, 64, generator=g, dtype=torch.float64)
    w = 1 + 0.2 * torch.randn(64, generator=g, dtype=torch.float64)
    th = ref.turns(torch.tensor([[[5, 900]]]), fa.rope_freqs(64), [32])
    dx, _, dw, _ = ref.norm_rope_bwd(dy, x, w, th, True, True, 1e-3)
    f = lambda x, w: float((ref.norm_rope(x, w, th, True, True, 1e-3)[0] * dy).sum())
    for i in (0, 1, 17, 63):
        e = torch.zeros_like(x)
        e[0, 0, 1, i] = 1e-6
        assert abs((f(x + e, w) - f(x - e, w)) / 2e-6 - float(dx[0, 0, 1, i])) < 1e-7
        assert abs((f(x, w + e[0, 0, 1]) - f(x, w - e[0, 0, 1])) / 2e-6 - float(dw[i])) < 1e-7


def test_empty(fa):
    e = torch.zeros((0, 4, 5, 64), device="cuda", dtype=torch.bfloat16)
    z = torch.zeros((2, 4, 0, 64), device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda")
    for x in (e, z):
        a, b = fa.qk_norm_rope(x, x, q_weight=w)
        assert a.shape == x.shape and b.shape == x.shape
        out = fa.qk_norm_rope_bwd(x, x, x, x, q_weight=w, k_weight=w)
        assert (out[2] == 0).all() and (out[3] == 0).all()
    fa.sync_status()


def test_streams_and_graph(fa):
    """Another stream, and a captured call replayed on new inputs."""
    q, k, w, pos, g = make(2, 8, 2, 50, 128, fused=False)
    freqs = fa.rope_freqs(128)
    dy = [torch.randn(x.shape, generator=g, device="cuda") for x in (q, k)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fa.qk_norm_rope(q, k, pos, freqs, *w)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = fa.qk_norm_rope(q, k, pos, freqs, *w)
            d = fa.qk_norm_rope_bwd(*dy, q, k, pos, freqs, *w)
    torch.cuda.current_stream().wait_stream(side)
    q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
    pos += 11
    graph.replay()
    graph.replay()
    for a, b in zip((*y, *d), (*fa.qk_norm_rope(q, k, pos, freqs, *w), *fa.qk_norm_rope_bwd(*dy, q, k, pos, freqs, *w))):
        assert torch.equal(a, b)


def test_refusals(fa):
    q, k, w, pos, _ = make(1, 2, 2, 8, 64)
    f = fa.rope_freqs(64)
    for args, kw in (((q, k, pos), {}), ((q, k, None, f), {}), ((q, k, pos, f.float()), {}), ((q, k, pos, f.cuda()), {}),
                     ((q, k, pos.long(), f), {}), ((q, k, pos, f), dict(sections=(16, 15))),
                     ((q, k, pos, f), dict(sections=(16, 16))), ((q, k, pos, f), dict(sections=(32, 0, 0, 0, 0))),
                     ((q, k, pos, f, w[0], w[1].to(torch.bfloat16)), {}), ((q, k, pos, f, w[0]), dict(norm=False)),
                     ((q, k), dict(norm=False)), ((q, None, pos, f, None, w[0]), {}), ((q, k[:, :, :7], pos, f), {}),
                     ((q.float(), k, pos, f), {})):
        with pytest.raises(ValueError):
            fa.qk_norm_rope(*args, **kw)
    with pytest.raises(fa.api.Fa4Fp4Error):
        fa.qk_norm_rope(q, k, pos, f, eps=-1.0)
    odd = torch.empty(1 * 8 * 2 * 64 + 4, device="cuda", dtype=torch.bfloat16)[4:].view(1, 2, 8, 64)
    with pytest.raises(fa.api.Fa4Fp4Error):
        fa.qk_norm_rope(odd, k, pos, f)
    dy = [x.contiguous() for x in (q, k)]
    with pytest.raises(ValueError):
        fa.qk_norm_rope_bwd(dy[0], dy[1].float(), q, k, pos, f)
    with pytest.raises(fa.api.Fa4Fp4Error):
        fa.qk_norm_rope_bwd(*dy, q, k, pos, f, *w, workspace=torch.empty(16, device="cuda", dtype=torch.uint8))
    ws = torch.empty(fa.qk_norm_rope_bwd_workspace_bytes(1, 2, 2, 8, 64), device="cuda", dtype=torch.uint8)
    for a, b in zip(fa.qk_norm_rope_bwd(*dy, q, k, pos, f, *w, workspace=ws), fa.qk_norm_rope_bwd(*dy, q, k, pos, f, *w)):
        assert torch.equal(a, b)
    fa.sync_status()


def test_far_offsets(fa):
    """Element offsets that pass 32 bits."""
    room = torch.empty(2 ** 31 + 2 ** 20, device="cuda", dtype=torch.bfloat16)
    q, k = (room[at:].as_strided((2, 2, 100, 64), (2 ** 31, 6400, 64, 1)) for at in (0, 2 ** 16))
    q0, k0, w, pos, _ = make(2, 2, 2, 100, 64, fused=False)
    q.copy_(q0)
    k.copy_(k0)
    f = fa.rope_freqs(64)
    assert all(torch.equal(a, b) for a, b in zip(fa.qk_norm_rope(q, k, pos, f, *w), fa.qk_norm_rope(q0, k0, pos, f, *w)))
    out = fa.qk_norm_rope_bwd(q0, k0, q, k, pos, f, *w, dq=q, dk=k)
    assert all(torch.equal(a, b) for a, b in zip(out, fa.qk_norm_rope_bwd(q0, k0, q0, k0, pos, f, *w)))


@pytest.mark.parametrize("f32", [False, True])
def test_backward_in_place(fa, f32):
    """dq in q's place, and dk in k's: more tokens than the GPU has warps."""
    q, k, w, pos, g = make(3, 6, 2, 5000, 64)
    freqs = fa.rope_freqs(64)
    dy = [torch.randn(x.shape, generator=g, device="cuda").to(torch.float32 if f32 else torch.bfloat16) for x in (q, k)]
    want = fa.qk_norm_rope_bwd(*dy, q, k, pos, freqs, *w)
    got = fa.qk_norm_rope_bwd(*dy, q, k, pos, freqs, *w, dq=q, dk=k)
    assert got[0] is q and got[1] is k
    assert all(torch.equal(a, b) for a, b in zip(got, want))
