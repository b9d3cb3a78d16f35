"""Norm and rotation, and cross attention, at the ends of what their calls allow."""
import math

import pytest
import torch

import layer_ref as ref
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def fa():
    return require_gpu()


def make(B, Hq, Hkv, Nq, Nk, d, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda H, N: torch.randn((B, H, N, d), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    return new(Hq, Nq), new(Hkv, Nk), new(Hkv, Nk), new(Hq, Nq)


def check_fwd(fa, q, k, v):
    o, lse = fa.cross_fwd(q, k, v)
    want, bound, wl, bl = ref.cross(q, k, v)
    ref.assert_within(o, want, bound, "o")
    ref.assert_within(lse, wl, bl, "lse")
    return o, lse


# query heads that share a tile and do not fill their kv head's last one
SHARED = [(1, 14, 2, 20, 300), (2, 21, 3, 33, 129), (1, 10, 2, 64, 64), (2, 14, 2, 1, 40), (1, 12, 4, 50, 1000)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk", SHARED)
def test_gradients_of_tiles_not_filled(fa, d, B, Hq, Hkv, Nq, Nk):
    q, k, v, dout = make(B, Hq, Hkv, Nq, Nk, d)
    o, lse = check_fwd(fa, q, k, v)
    for name, x, (want, bound) in zip(("dq", "dk", "dv"), fa.cross_bwd(q, k, v, o, dout, lse),
                                      ref.cross_bwd(q, k, v, o, dout, lse)):
        ref.assert_within(x, want, bound, name)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), INF, 3e38])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk", SHARED)
def test_kv_heads_stay_apart(fa, d, bad, B, Hq, Hkv, Nq, Nk):
    """What is not finite in one kv head, its queries or their gradients, changes nothing in the others."""
    q, k, v, dout = make(B, Hq, Hkv, Nq, Nk, d)
    G = Hq // Hkv
    o, lse = fa.cross_fwd(q, k, v)
    want = fa.cross_bwd(q, k, v, o, dout, lse)
    for h in (1, Hkv - 1):
        q2, k2, v2, g2 = (x.clone() for x in (q, k, v, dout))
        others = [x for x in range(Hkv) if x != h]
        heads = [x for x in range(Hq) if x // G != h]
        for x in (q2, g2):
            x[:, h * G: (h + 1) * G, ::3] = bad
        k2[:, h, ::2], v2[:, h, 1::2] = bad, bad
        for a, b, e in ((q2, k2, g2), (q2, k, dout), (q, k, g2)):
            o2, lse2 = fa.cross_fwd(a, b, v2)
            assert torch.equal(o2[:, heads], o[:, heads]) and torch.equal(lse2[:, heads], lse[:, heads])
            dq, dk, dv = fa.cross_bwd(a, b, v2, o2, e, lse2)
            assert torch.equal(dq[:, heads], want[0][:, heads])
            assert torch.equal(dk[:, others], want[1][:, others]) and torch.equal(dv[:, others], want[2][:, others])
    fa.sync_status()


@pytest.mark.parametrize("B,H,N,axes", [(64, 8, 1, 1), (2, 4, 600, 3)])
def test_positions_of_the_launch_before(fa, B, H, N, axes):
    """Positions, weights and rows that the launch right before the call writes, over and over."""
    d = 128
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((B, H, N, d), generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn((B, H, N, d), generator=g, device="cuda").to(torch.bfloat16)
    sections = [d // 2 - (axes - 1) * (d // 2 // axes)] + [d // 2 // axes] * (axes - 1)
    freqs = fa.rope_freqs(d, sections)
    start = torch.randint(0, 1000, (B, axes, N), generator=g, device="cuda").int()
    steps = 60
    want = []
    for i in range(steps):
        pos = start + 7 * i
        torch.cuda.synchronize()
        want.append((fa.qk_norm_rope(x, None, pos, freqs, sections=sections)[0],
                     fa.qk_norm_rope_bwd(dy, None, x, None, pos, freqs, sections=sections)[0]))
        torch.cuda.synchronize()
    pos = start.clone()

    def run():
        got = []
        for i in range(steps):
            y = fa.qk_norm_rope(x, None, pos, freqs, sections=sections)[0]
            got.append((y, fa.qk_norm_rope_bwd(dy, None, x, None, pos, freqs, sections=sections)[0]))
            pos.add_(7)
        return got

    eager = run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for _ in range(5):
        pos.copy_(start)
        graph.replay()
        for got in (eager, captured):
            for a, b in zip(want, got):
                assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [3, 200])
@pytest.mark.parametrize("Nk", [1, 100, 1000, 6000])
def test_values_near_the_end(fa, d, Nq, Nk):
    """Values up to the largest of bf16, whose sums before the division would pass FP32's, and very small ones."""
    q, k, v, _ = make(1, 4, 2, Nq, Nk, d)
    most = torch.finfo(torch.bfloat16).max
    u = torch.rand(v.shape, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    q[:, :, 0] = 0                                     # a row of equal weights
    for values in ((0.5 + 0.5 * u) * most, torch.full_like(u, most), v.float() / 8 * most):
        values = values.to(torch.bfloat16)
        values = torch.where(values.isinf(), torch.full_like(values, most), values)
        check_fwd(fa, q, k, values)
        check_fwd(fa, q, k, (values.float() * 2.0 ** -228).to(torch.bfloat16))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [3, 200, 700])
@pytest.mark.parametrize("Nk,lost", [(300, 128), (1000, 900), (40, 32)])
def test_scores_past_the_range(fa, d, Nq, Nk, lost):
    """Scores that pass FP32's range below, in the first keys: those keys have no weight, the others all of it."""
    q, k, v, dout = make(1, 2, 2, Nq, Nk, d)
    q[..., 0] = 1e20
    k[..., 0] = 0
    k[:, :, :lost] = 0
    k[:, :, :lost, 0] = -1e20
    q[..., 1:] = 1.0
    k[:, :, lost:, 1:] -= 30.0                         # scores of some hundred below zero
    o, lse = fa.cross_fwd(q, k, v)
    want, bound, wl, bl = ref.cross(q, k[:, :, lost:], v[:, :, lost:])
    ref.assert_within(o, want, bound, "o")
    ref.assert_within(lse, wl, bl, "lse")
    dq, dk, dv = fa.cross_bwd(q, k, v, o, dout, lse)
    assert (dk[:, :, :lost] == 0).all() and (dv[:, :, :lost] == 0).all()
    assert torch.isfinite(dq).all() and torch.isfinite(dk).all() and torch.isfinite(dv).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [3, 200, 700])
@pytest.mark.parametrize("Nk", [20, 300])
def test_no_score_within_the_range(fa, d, Nq, Nk):
    """All scores of a row past FP32's range below: as a row without a key."""
    q, k, v, dout = make(1, 2, 2, Nq, Nk, d)
    q[:, :, 1] = 0
    q[:, :, 1, 0] = 1e20
    k[..., 0] = -1e20
    q[:, :, [0, 2], 0] = 0
    o, lse = fa.cross_fwd(q, k, v)
    assert (lse[:, :, 1] == -INF).all() and (o[:, :, 1] == 0).all()
    want, bound, wl, bl = ref.cross(q[:, :, [0, 2]], k, v)
    ref.assert_within(o[:, :, [0, 2]], want, bound, "o")
    dq = fa.cross_bwd(q, k, v, o, dout, lse)[0]
    assert (dq[:, :, 1] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nk", [(2, 20), (2, 5000), (40, 60), (300, 500)])
def test_rows_that_are_not_finite(fa, d, Nq, Nk):
    """A query that is not finite has neither o nor lse, and is no row without a key; the others are as they were."""
    q, k, v, _ = make(2, 4, 2, Nq, Nk, d)
    lens = torch.tensor([Nk, 0], device="cuda", dtype=torch.int32)
    o, lse = fa.cross_fwd(q, k, v, lens)
    q[:, 1, 0] = float("nan")
    q[:, 2, 1, 3] = INF
    o2, lse2 = fa.cross_fwd(q, k, v, lens)
    bad = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    bad[0, 1, 0] = bad[0, 2, 1] = True
    assert lse2[bad].isnan().all() and o2[bad].isnan().all()
    assert torch.equal(lse2[~bad], lse[~bad]) and torch.equal(o2[~bad], o[~bad])
    assert (lse2[1] == -INF).all() and (o2[1] == 0).all()


def test_no_query_heads(fa):
    """Keys that no head attends to have gradients of zeros."""
    q = torch.zeros((2, 0, 5, 64), device="cuda", dtype=torch.bfloat16)
    k = torch.ones((2, 3, 9, 64), device="cuda", dtype=torch.bfloat16)
    o, lse = fa.cross_fwd(q, k, k)
    outs = [torch.full_like(k, 7.0) for _ in range(2)]
    dq, dk, dv = fa.cross_bwd(q, k, k, o, q, lse, dk=outs[0], dv=outs[1])
    assert o.shape == dq.shape == q.shape and (dk == 0).all() and (dv == 0).all()
    fa.sync_status()


def turn_exactly(freq):
    """The angle of a position, position * freq modulo 2 pi, in whole numbers."""
    two_pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239)) * 2      # times 2^BITS (Machin)
    num, den = freq.as_integer_ratio()
    return lambda p: ((p * num << BITS) // den % two_pi) / (1 << BITS)


BITS = 200


def arctan_inverse(n):
    total = term = (1 << BITS) // n
    i, sign = 3, -1
    while term:
        term //= n * n
        total += sign * (term // i)
        i, sign = i + 2, -sign
    return total


def test_exact_turns():
    assert abs(turn_exactly(1.0)(7) - math.fmod(7.0, 2 * math.pi)) < 1e-15
    assert abs(turn_exactly(0.5)(-1) - (2 * math.pi - 0.5)) < 1e-15


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions_of_high_frequencies(fa, interleaved):
    """Angles do not worsen with the position.  A sine or cosine is off by 3.0e-7 for its angle's roundings to FP32 and by
    2^-21.2 for the native function, the sum of two products by another 1.2e-7 of their sizes: below 2^-20 of them."""
    d, N, H = 64, 512, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((1, H, N, d), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.randint(2 ** 31 - 2 ** 20, 2 ** 31, (1, 1, N), generator=g, device="cuda").int()
    pos[:, :, ::2] *= -1
    freqs = torch.linspace(-2 * math.pi, 2 * math.pi, d // 2 + 1, dtype=torch.float64)[1:] * 0.999
    freqs[0], freqs[1] = 1e-9, 1e6 + 0.37
    places = pos[0, 0].tolist()
    th = torch.stack([torch.tensor([t(p) for p in places], dtype=torch.float64)
                      for t in (turn_exactly(float(f)) for f in freqs)], -1)[None, None].cuda()
    y, _ = fa.qk_norm_rope(x, None, pos, freqs, norm=False, interleaved=interleaved)
    want = ref.turn(x.double(), th, interleaved)
    a, b = ref.split(x.double().abs(), interleaved)
    ref.assert_within(y, want, ref.U * want.abs() + 2.0 ** -20 * ref.join(a + b, a + b, interleaved), "q")


class Watch(torch.utils._python_dispatch.TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.shapes = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func is torch.ops.aten.empty.memory_format:
            self.shapes.append(tuple(out.shape))
        return out


def test_outputs_are_seen_by_torch(fa):
    """The tensors that a call makes go through torch's dispatcher where something there looks at them: a dispatch mode, or
    the filling of uninitialised memory."""
    q, k, v, dout = make(1, 2, 2, 4, 8, 64)
    cache = fa.cache_alloc(1, 2, 64, page=16)
    table = torch.zeros((1, 1), device="cuda", dtype=torch.int32)
    lens = torch.zeros(1, device="cuda", dtype=torch.int32)
    fa.cache_append(cache, k, v, table, lens)
    lens += 8

    def calls():
        o, lse = fa.cross_fwd(q, k, v)
        return (o, lse, *fa.cross_bwd(q, k, v, o, dout, lse), *fa.qk_norm_rope(q, dout),
                *fa.cache_fwd(q, cache, table, lens))

    want = calls()
    with Watch() as seen:
        got = calls()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    for x in want:
        assert tuple(x.shape) in seen.shapes
    assert sum(s == tuple(q.shape) for s in seen.shapes) >= 4
    was = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)
    try:
        assert torch.utils.deterministic.fill_uninitialized_memory
        with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as prof:
            got = calls()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    finally:
        torch.use_deterministic_algorithms(was)
    fills = sum(e.count for e in prof.key_averages() if e.key == "aten::fill_")
    assert fills >= len(want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_of_every_size(fa, d, interleaved, eps):
    """Rows whose squares pass FP32's range at either end, beside others, and rows of large and small channels."""
    g = torch.Generator(device="cuda").manual_seed(7)
    B, H, N = 2, 5, 9
    new = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    sizes = torch.tensor([0, 126, 100, 64, 60, 51, 40, -40, -60, -75, -100, -120], device="cuda").float()
    if eps:
        sizes = sizes.clamp(min=0)
    rows = 2.0 ** sizes[torch.randint(0, 12, (B, H, N, 1), generator=g, device="cuda")]
    x = (new(B, H, N, d).clamp(-1.9, 1.9) * rows).to(torch.bfloat16)
    x[0, 0, :, : d // 4] *= 2.0 ** -30
    w = 1 + 0.2 * new(d)
    pos = torch.randint(0, 5000, (B, 1, N), generator=g, device="cuda").int()
    freqs = fa.rope_freqs(d)
    th = ref.turns(pos, freqs, [d // 2])
    y, _ = fa.qk_norm_rope(x, None, pos, freqs, w, interleaved=interleaved, eps=eps)
    ref.assert_within(y, *ref.norm_rope(x, w, th, interleaved, True, eps), "y")
    dy = new(B, H, N, d)
    for dt in (torch.float32, torch.bfloat16):
        dx, _, dw, _ = fa.qk_norm_rope_bwd(dy.to(dt), None, x, None, pos, freqs, w, interleaved=interleaved, eps=eps)
        want, bound, want_w, bound_w = ref.norm_rope_bwd(dy.to(dt), x, w, th, interleaved, True, eps)
        ref.assert_within(dx, want, bound, "dx")
        ref.assert_within(dw, want_w, bound_w, "dw")


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_of_every_size_in_place(fa, f32, eps):
    """Gradients in their rows' places, among which are rows beyond FP32's squares and others whose gradients are far too
    small or large: what a row's place holds by then is not taken for the row."""
    g = torch.Generator(device="cuda").manual_seed(8)
    B, H, N, d = 2, 150, 40, 64
    new = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    sizes = torch.tensor([0, 0, 0, 100, -40, 45] + ([-70] if eps == 0 else [60]), device="cuda").float()
    x = (new(B, H, N, d) * 2.0 ** sizes[torch.randint(0, 7, (B, H, N, 1), generator=g, device="cuda")]).to(torch.bfloat16)
    dy = new(B, H, N, d) * 2.0 ** sizes[torch.randint(0, 6, (B, H, N, 1), generator=g, device="cuda")].clamp(-60, 45)
    dy[:, ::5] = 0.0
    dy = dy.to(torch.float32 if f32 else torch.bfloat16)
    w = 1 + 0.2 * new(d)
    pos = torch.randint(0, 5000, (B, 1, N), generator=g, device="cuda").int()
    args = (pos, fa.rope_freqs(d), w)
    want = fa.qk_norm_rope_bwd(dy, None, x, None, *args, eps=eps)
    dx, bound, _, _ = ref.norm_rope_bwd(dy, x, w, ref.turns(pos, args[1], [d // 2]), False, True, eps)
    ref.assert_within(want[0], dx, bound, "dx")
    got = fa.qk_norm_rope_bwd(dy, None, x, None, *args, eps=eps, dq=x)
    assert got[0] is x and torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    y = fa.qk_norm_rope(x, None, *args, eps=1e-6)[0]
    assert torch.equal(fa.qk_norm_rope(x, None, *args, eps=1e-6, q_out=x)[0], y)


@pytest.mark.parametrize("d,H", [(64, 300), (128, 131)])
def test_many_heads_of_many_tokens(fa, d, H):
    """More heads than a warp takes at a time, with tokens enough for every warp; every row of some tokens beyond FP32's
    squares."""
    g = torch.Generator(device="cuda").manual_seed(9)
    N = 3001
    x = torch.randn((1, N, H, d), generator=g, device="cuda")
    x[:, 5::700] *= 2.0 ** 70
    x = x.to(torch.bfloat16).transpose(1, 2)
    dy = torch.randn((1, N, H, d), generator=g, device="cuda").to(torch.bfloat16).transpose(1, 2)
    w = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
    pos = torch.arange(N, device="cuda", dtype=torch.int32)[None]
    freqs = fa.rope_freqs(d)
    th = ref.turns(pos[None], freqs, [d // 2])
    y, _ = fa.qk_norm_rope(x, None, pos, freqs, w)
    dx, _, dw, _ = fa.qk_norm_rope_bwd(dy, None, x, None, pos, freqs, w)
    for h in range(0, H, 50):
        at = slice(h, min(H, h + 50))
        ref.assert_within(y[:, at], *ref.norm_rope(x[:, at], w, th, False, True, 1e-6), "y")
        want, bound, _, _ = ref.norm_rope_bwd(dy[:, at], x[:, at], w, th, False, True, 1e-6)
        ref.assert_within(dx[:, at], want, bound, "dx")
    parts = [ref.norm_rope_bwd(dy[:, h: h + 50], x[:, h: h + 50], w, th, False, True, 1e-6)[2:] for h in range(0, H, 50)]
    ref.assert_within(dw, sum(a for a, _ in parts), sum(b for _, b in parts), "dw")
