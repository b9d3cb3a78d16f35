"""The 8-bit cache at the ends of its range: runs of zero tokens, scales that
fall or rise by hundreds of powers of two, values close to the largest bf16.

The attention's bound is that of the other cache tests (weights and P relative,
the output's half step), but for what P loses as a f16 number: with U the unit of
128 keys (of a token's own list) and V_U its largest |v|, seen or not,

  |o - ref| <= (4 eps + 2^-19 + p_err) * spread + out_err * |ref|
               + 2^-35 * sum over U of 128 V_U e^min(0, M_U - m)

M_U being the largest score seen up to the end of U: a lost part of P shrinks with
everything else when a larger score comes later.  (A P times 2^15 and the ratio of
V's page scale to the accumulator's, at most 2^4 above that of its keys, is off by
half of f16's smallest step 2^-24: 2^-36 of a scale whose 448 is below 2 V_U.  2^12
and 2^1 in the kernel for many rows: the same.  An accumulator that holds values
more than 2^60 above is not brought down to a unit's own scale: that leaves 2^-96 of
those, which the terms of their own units contain.)"""
import numpy as np
import pytest
import torch

import cache_ref as R
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def queries(B, Hq, T, d, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, Hq, T, d, generator=g) * scale).to(torch.bfloat16).cuda()


def cache_of(fa, k, v, page, seed, first=0, stale=0xff):
    """A cache of the sequences k, v: [B][H, n_b, d] float tensors."""
    lens = [x.shape[1] for x in k]
    H, d = k[0].shape[0], k[0].shape[2]
    cache, table, ln = R.make(fa, lens, H, d, page, seed=seed, first=first, stale=stale)
    T = max(lens)
    pad = lambda xs: torch.stack([torch.nn.functional.pad(x, (0, 0, 0, T - x.shape[1])) for x in xs])
    fa.cache_append(cache, pad(k).bfloat16().cuda(), pad(v).bfloat16().cuda(), table, torch.zeros_like(ln), n_new=ln)
    return cache, table, ln, lens


def reference(ref, q, lens, T, f32, causal=True, scale=None, pages=None, heads=None):
    """o, lse and their bounds for T query tokens of every sequence (and the first
    `heads` kv heads)."""
    G, P = q.shape[1] // ref.H, ref.page
    q = q[:, :G * (heads or ref.H)]
    B, Hq, _, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    o, lse, tol = np.zeros(q.shape), np.full((B, Hq, T), -np.inf), np.zeros(q.shape)
    lse_tol = np.zeros((B, Hq, T))
    for b in range(B):
        L = int(lens[b])
        for hk in range(Hq // G):
            K, V = ref.read("k", b, hk, L), ref.read("v", b, hk, L)
            for t in range(T):
                n = ref.sees(L, T, t, causal)
                at = np.arange(L)
                if pages is not None:
                    at = np.concatenate([np.arange(p * P, min(p * P + P, L)) for p in pages[b, hk, t] if p >= 0] or [at[:0]])
                    unit = np.concatenate([np.arange(i * P, i * P + min(P, L - p * P)) // 128
                                           for i, p in enumerate(pages[b, hk, t]) if p >= 0] or [at[:0]])
                else:
                    unit = at // 128
                see = at < n
                if not see.any():
                    continue
                k, v = K[at], V[at]
                top = np.abs(v).max(1)
                for h in range(hk * G, hk * G + G):
                    s = np.where(see, k @ q[b, h, t] * scale, -np.inf)
                    m = s.max()
                    p = np.exp(s - m)
                    o[b, h, t] = p @ v / p.sum()
                    lse[b, h, t] = m + np.log(p.sum())
                    e = (np.abs(k) @ np.abs(q[b, h, t]))[see].max() * scale * d * 2.0 ** -23
                    lost, upto = 0.0, -np.inf
                    for u in np.unique(unit):
                        upto = max(upto, s[unit == u].max())
                        if upto > -np.inf:
                            lost += 2.0 ** -35 * 128 * top[unit == u].max() * np.exp(min(0.0, upto - m))
                    tol[b, h, t] = (4 * e + 2.0 ** -19 + (2.0 ** -22 if f32 else 2.0 ** -11)) * (p @ np.abs(v) / p.sum())
                    tol[b, h, t] += (2.0 ** -24 if f32 else 2.0 ** -8) * np.abs(o[b, h, t]) + lost + 1e-37
                    lse_tol[b, h, t] = 2 * e + 2.0 ** -20 + 2.0 ** -22 * abs(lse[b, h, t])
    return o, lse, tol, lse_tol


def check(fa, q, cache, table, ln, lens, f32, causal=True, scale=None, pages=None, heads=None):
    o, lse = fa.cache_fwd(q, cache, table, ln, causal=causal, softmax_scale=scale or 0.0, pages=pages,
                          out_dtype=fa.OUT_F32 if f32 else fa.OUT_BF16)
    fa.sync_status()
    ref = R.Ref.of(cache, table)
    want, wl, tol, lt = reference(ref, f64(q), lens, q.shape[2], f32, causal, scale,
                                  None if pages is None else pages.cpu().numpy(), heads)
    o, lse = f64(o[:, :wl.shape[1]]), f64(lse[:, :wl.shape[1]])
    assert np.isfinite(o).all()
    bad = np.abs(o - want) - tol
    assert bad.max() <= 0, f"o off by {bad.max():.3g} over its bound"
    seen = np.isfinite(wl)
    assert np.array_equal(np.isneginf(lse), ~seen) and not o[~seen].any()
    assert (np.abs(lse[seen] - wl[seen]) <= lt[seen]).all()


# ------------------------------------------------------------------ V's exponents, few rows
def zero_runs(H, d, seed, alike=1):
    """V is zero over 1, 2, 3 and 5 blocks of 128 tokens between others and at the
    end; and the same in sequences of few tokens.  `alike` times as many heads: with
    enough of them one CTA goes through several units of a head."""
    g = torch.Generator().manual_seed(seed)
    k, v = [], []
    for runs in ([128, -128, 128, -256, 100, -384, 130, -640, 60], [256, -1300], [-300, 200, -1024, 300, -700],
                 [3, -500], [-513], [16, -17, 5]):
        n = sum(abs(r) for r in runs)
        k.append(torch.randn(H, n, d, generator=g))
        x = torch.randn(H, n, d, generator=g)
        at = 0
        for r in runs:
            if r < 0:
                x[:, at:at - r] = 0
            at += abs(r)
        v.append(x)
    return [x.repeat(alike, 1, 1) for x in k], [x.repeat(alike, 1, 1) for x in v]


def falling(H, d, seed, first, last, keys, steps, alike=1):
    """|v| falls (or rises) from 2^first to 2^last in equal steps of `keys` tokens."""
    g = torch.Generator().manual_seed(seed)
    n = keys * steps
    k = torch.randn(H, n, d, generator=g)
    v = torch.randn(H, n, d, generator=g)
    for i in range(steps):
        v[:, i * keys:(i + 1) * keys] *= 2.0 ** (first + (last - first) * i / max(steps - 1, 1))
    return [k.repeat(alike, 1, 1)], [v.repeat(alike, 1, 1)]


FEW = [(64, 16, 2, 3, 1, False), (64, 64, 1, 1, 5, True), (128, 32, 2, 4, 1, False), (128, 128, 1, 3, 4, True),
       (128, 16, 1, 2, 8, False), (64, 128, 2, 4, 16, False), (128, 64, 1, 1, 1, True)]


@pytest.mark.parametrize("alike", [1, 60])
@pytest.mark.parametrize("d,page,H,G,T,f32", FEW)
def test_fwd_runs_of_zero_v(d, page, H, G, T, f32, alike):
    fa = require_gpu()
    k, v = zero_runs(H, d, 1, alike)
    cache, table, ln, lens = cache_of(fa, k, v, page, 2)
    q = queries(len(lens), H * alike * G, T, d, 3)
    for causal in (True, False):
        check(fa, q, cache, table, ln, lens, f32, causal, heads=H)
    sel = fa.cache_select(q, cache, table, ln, 700 // page + 1)
    check(fa, q, cache, table, ln, lens, f32, pages=sel, heads=H)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("first,last", [(100, -100), (-100, 100), (70, -126), (0, -120)])
@pytest.mark.parametrize("T,keys,steps,alike", [(1, 128, 5, 1), (1, 128, 5, 240), (3, 256, 9, 1), (2, 256, 9, 240),
                                                (1, 640, 2, 240), (12, 64, 21, 1), (4, 64, 21, 240)])
def test_fwd_v_falls_and_rises(T, keys, steps, alike, first, last, f32):
    fa = require_gpu()
    d, page, G = 128, 32, 4
    k, v = falling(1, d, 4, first, last, keys, steps, alike)
    cache, table, ln, lens = cache_of(fa, k, v, page, 5)
    q = queries(1, alike * G, T, d, 6)
    check(fa, q, cache, table, ln, lens, f32, heads=1)
    all_pages = torch.arange(table.shape[1], dtype=torch.int32, device="cuda").expand(1, alike, T, -1).contiguous()
    check(fa, q, cache, table, ln, lens, f32, pages=all_pages, heads=1)


@pytest.mark.parametrize("T,f32", [(1, True), (1, False), (4, True), (4, False)])
def test_fwd_large_v_without_weight(T, f32):
    """Far larger values whose weight a later score takes away from some of the
    rows only: those rows' small values keep their accuracy, the others theirs."""
    fa = require_gpu()
    d, page, H, G, n = 64, 16, 480, 4, 1700
    g = torch.Generator().manual_seed(7)
    k = (torch.randn(1, n, d, generator=g) * 0.1).repeat(H, 1, 1)
    v = torch.randn(1, n, d, generator=g).repeat(H, 1, 1)
    v[:, :300] *= 2.0 ** 100
    v[:, 300:800] *= 2.0 ** 40
    v[:, 1200:] *= 2.0 ** -30
    k[:, 800:, 0] = 60.0                  # scores 60 q_0: 0 or 300
    cache, table, ln, lens = cache_of(fa, [k], [v], page, 8)
    q = queries(1, H * G, T, d, 9)
    q[:, :, :, 0] = 0
    q[:, ::2, :, 0] = 5
    check(fa, q, cache, table, ln, lens, f32, scale=1.0, heads=1)


# ------------------------------------------------------------------ V's exponents, many rows
@pytest.mark.parametrize("d,page,H,G,T", [(64, 16, 2, 3, 40), (128, 64, 1, 2, 200), (128, 16, 1, 4, 70), (64, 128, 1, 1, 300)])
def test_fwd_chunk_runs_of_zero_v(d, page, H, G, T):
    fa = require_gpu()
    k, v = zero_runs(H, d, 11)
    cache, table, ln, lens = cache_of(fa, k, v, page, 12)
    q = queries(len(lens), H * G, T, d, 13)
    for causal in (True, False):
        check(fa, q, cache, table, ln, lens, False, causal)
    check(fa, q, cache, table, ln, lens, True)


@pytest.mark.parametrize("first,last", [(100, -100), (-100, 100), (70, -126), (0, -120)])
@pytest.mark.parametrize("d,T,keys,steps", [(128, 70, 128, 5), (64, 80, 256, 9), (128, 65, 640, 2), (64, 200, 64, 21)])
def test_fwd_chunk_v_falls_and_rises(d, T, keys, steps, first, last):
    fa = require_gpu()
    k, v = falling(1, d, 14, first, last, keys, steps)
    cache, table, ln, lens = cache_of(fa, k, v, 32, 15)
    q = queries(1, 2, T, d, 16)
    check(fa, q, cache, table, ln, lens, False)


@pytest.mark.parametrize("d", [64, 128])
def test_fwd_chunk_large_v_without_weight(d):
    """As above: 70 rows of a head side by side, every second of which loses the
    large values' weight."""
    fa = require_gpu()
    page, H, G, T, n = 64, 1, 2, 70, 1700
    g = torch.Generator().manual_seed(17)
    k = torch.randn(H, n, d, generator=g) * 0.1
    v = torch.randn(H, n, d, generator=g)
    v[:, :300] *= 2.0 ** 100
    v[:, 300:800] *= 2.0 ** 40
    v[:, 1200:] *= 2.0 ** -30
    k[:, 800:, 0] = 60.0
    cache, table, ln, lens = cache_of(fa, [k], [v], page, 18)
    q = queries(1, H * G, T, d, 19)
    q[..., 0] = 0
    q[:, :, ::2, 0] = 5
    check(fa, q, cache, table, ln, lens, False, scale=1.0)


# ------------------------------------------------------------------ small queries, zero keys, many rows
@pytest.mark.parametrize("d,page,H,G,T,scale", [(128, 64, 2, 2, 70, None), (64, 16, 1, 3, 100, None), (128, 128, 1, 1, 90, 1e-12),
                                                (64, 32, 2, 1, 66, 1e-6)])
def test_fwd_chunk_small_queries(d, page, H, G, T, scale):
    """Pool page 0 unused, its scale byte 0 (2^-127), keys that end inside a tile, and
    pages of zero keys at the causal edge: rows of q down to the smallest bf16."""
    fa = require_gpu()
    g = torch.Generator().manual_seed(21)
    lens = [T + 5, 3 * T + 1, 128, 7, 300]
    k = [torch.randn(H, n, d, generator=g) for n in lens]
    k[1][:, 2 * T:] = 0
    k[4][:] = 0
    k[2][:, 100:] *= 2.0 ** -120
    v = [torch.randn(H, n, d, generator=g) for n in lens]
    cache, table, ln, lens = cache_of(fa, k, v, page, 22, first=1)
    assert int(cache.ks[0].max()) == 0 and int(table.min()) > 0
    q = queries(len(lens), H * G, T, d, 23)
    q *= (2.0 ** -(torch.arange(T) % 14 * 10).float()).view(1, 1, T, 1).cuda()      # down to 2^-130
    for causal in (True, False):
        check(fa, q, cache, table, ln, lens, False, causal, scale)


# ------------------------------------------------------------------ V close to the largest bf16
@pytest.mark.parametrize("d,page,H,G,T,f32", FEW + [(128, 64, 1, 2, 70, False), (64, 16, 1, 3, 90, False), (64, 16, 1, 3, 90, True)])
def test_fwd_largest_values(d, page, H, G, T, f32):
    """A mean of values up to 2^127.99 is one itself; so are keys of nearly equal
    weight in great number, and a row whose keys are cut among CTAs."""
    fa = require_gpu()
    g = torch.Generator().manual_seed(31)
    big = float(torch.finfo(torch.bfloat16).max)
    lens = [1, 40, 513, 6000]
    k = [torch.randn(H, n, d, generator=g) * 0.01 for n in lens]
    v = [torch.rand(H, n, d, generator=g) * 0.9 * big for n in lens]
    for x in v:
        x[:, :, ::2] *= -1
        x[:, :, 1] *= 2.0 ** -30
    cache, table, ln, lens = cache_of(fa, k, v, page, 32)
    q = queries(len(lens), H * G, T, d, 33)
    check(fa, q, cache, table, ln, lens, f32)
    small = [x * 2.0 ** -200 for x in v]
    cache, table, ln, lens = cache_of(fa, k, small, page, 34)
    check(fa, q, cache, table, ln, lens, f32)


# ------------------------------------------------------------------ received weights
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (64, 128)])
@pytest.mark.parametrize("G,T", [(1, 1), (4, 4), (4, 10), (4, 40)])
def test_weigh_bad_page(d, page, G, T):
    """The keys of a page that is not in the pool receive nothing; their old
    weights arrive all the same, in every kernel."""
    fa = require_gpu()
    H, lens = 2, [3 * page + 5, 300, 2 * page]
    cache, table, ln = R.make(fa, lens, H, d, page, seed=25)
    q = queries(3, H * G, T, d, 26)
    ql = torch.tensor([T, T, 0], dtype=torch.int32).cuda()
    _, lse = fa.cache_fwd(q, cache, table, ln, q_lens=ql, out_dtype=fa.OUT_F32)
    w = torch.rand(3, H, table.shape[1] * page, device="cuda")
    good, out = torch.full_like(w, 5.0), torch.full_like(w, 5.0)
    fa.cache_weigh(q, lse, cache, table, ln, w, q_lens=ql, out=good)
    fa.sync_status()
    bad = table.clone()
    bad[0, 1], bad[1, 0], bad[2, 1] = cache.num_pages, -1, 1 << 30
    fa.cache_weigh(q, lse, cache, bad, ln, w, q_lens=ql, out=out)
    with pytest.raises(fa.Fa4Fp4Error) as e:
        fa.sync_status()
    assert e.value.status == 7
    for b, p in ((0, 1), (1, 0), (2, 1)):
        at = slice(p * page, min((p + 1) * page, lens[b]))
        assert torch.equal(out[b, :, at], w[b, :, at])
        good[b, :, at] = w[b, :, at]
    assert torch.equal(out, good)


WEIGH = [(64, 16, 1, 7), (128, 64, 2, 8), (128, 32, 2, 20), (64, 128, 1, 79), (128, 64, 2, 100)]


def weigh_with(fa, d, page, G, T, value):
    """Weights with one row's lse set to `value`, and with the row left out."""
    H, lens = 2, [T + 150, T, 129]
    cache, table, ln = R.make(fa, lens, H, d, page, seed=27)
    q = queries(3, H * G, T, d, 28)
    _, lse = fa.cache_fwd(q, cache, table, ln, out_dtype=fa.OUT_F32)
    w = torch.rand(3, H, table.shape[1] * page, device="cuda")
    t = T // 2
    none, some = lse.clone(), lse.clone()
    none[:, 0, t] = float("-inf")
    some[:, 0, t] = value
    want = fa.cache_weigh(q, none, cache, table, ln, w, out=w.clone())
    got = fa.cache_weigh(q, some, cache, table, ln, w, out=w.clone())
    fa.sync_status()
    return got, want, [max(0, min(n, n - T + t + 1)) for n in lens]


@pytest.mark.parametrize("d,page,G,T", WEIGH)
def test_weigh_row_of_nan(d, page, G, T):
    """A token whose lse is not a number says nothing about the keys that it does
    not see."""
    got, want, sees = weigh_with(require_gpu(), d, page, G, T, float("nan"))
    for b, n in enumerate(sees):
        assert torch.isnan(got[b, 0, :n]).all()
        assert torch.equal(got[b, 0, n:], want[b, 0, n:]) and torch.equal(got[b, 1:], want[b, 1:])


@pytest.mark.parametrize("d,page,G,T", WEIGH)
def test_weigh_row_of_infinite_lse(d, page, G, T):
    """e^(s - inf) = 0 for every key."""
    got, want, _ = weigh_with(require_gpu(), d, page, G, T, float("inf"))
    assert torch.equal(got, want)


# ------------------------------------------------------------------ calls from several threads
def test_select_from_two_threads():
    """Tables of different lengths at once, each on its own stream: the kernel's
    limit of shared memory is one for the whole process."""
    import threading
    fa = require_gpu()
    d, page, H = 64, 16, 1
    caches = [R.make(fa, [n], H, d, page, seed=35, room=room) for n, room in ((5000, 16 * 9000), (5000, 16 * 16000))]
    q = queries(1, 2, 1, d, 36)
    want = [fa.cache_select(q, c, t, ln, 20) for c, t, ln in caches]
    fa.sync_status()
    errors = []

    def run(i):
        try:
            c, t, ln = caches[i]
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(3000):
                    got = fa.cache_select(q, c, t, ln, 20)
                torch.cuda.current_stream().synchronize()
                assert torch.equal(got, want[i])
        except BaseException as e:
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i % 2,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    fa.sync_status()
    assert not errors, errors


# ------------------------------------------------------------------ status
def test_every_kind_of_error_is_reported():
    """Errors of different kinds between two looks at the status: each is
    reported, the more serious first, and then none."""
    fa = require_gpu()
    cache, table, ln = R.make(fa, [0, 0], 2, 64, 16, room=20)
    zero = torch.zeros_like(ln)
    x = queries(2, 2, 3, 64, 37)
    x[0, 0, 1, 5] = float("nan")
    bad = table.clone()
    bad[1, 0] = -1
    fa.sync_status()
    fa.watchdog_selftest(1_000_000)
    fa.cache_append(cache, x, x, bad, zero)
    fa.cache_append(cache, x, x, bad, zero)
    for status in (5, 7, 8):
        with pytest.raises(fa.Fa4Fp4Error) as e:
            fa.sync_status()
        assert e.value.status == status
    fa.sync_status()


# ------------------------------------------------------------------ the cache's tensors
def test_cache_tensors_with_other_memory():
    """A call uses the memory that the cache's tensors have then, and refuses
    tensors that have lost the cache's shape."""
    fa = require_gpu()
    cache, table, ln = R.make(fa, [40, 70], 2, 64, 16, seed=40)
    q = queries(2, 4, 1, 64, 41)
    want = fa.cache_fwd(q, cache, table, ln)[0]
    old = {n: getattr(cache, n).clone() for n in ("k", "v", "ks", "vs", "kb")}
    for name in old:
        t = getattr(cache, name)
        t.set_(t.clone())
    fa.sync_status()
    for name in old:
        getattr(cache, name).copy_(old[name])
    assert torch.equal(fa.cache_fwd(q, cache, table, ln)[0], want)
    zero = torch.zeros_like(ln)
    new = queries(2, 2, 3, 64, 42)
    fa.cache_append(cache, new, new, table, zero)
    assert not torch.equal(cache.k, old["k"])              # stored in the new memory
    for name, t in old.items():
        getattr(cache, name).copy_(t)
    v = cache.v
    for change in (lambda: v.set_(v[:-1].clone()), lambda: v.set_(old["v"].transpose(2, 3))):
        change()
        with pytest.raises(ValueError, match="v: expected"):
            fa.cache_fwd(q, cache, table, ln)
        with pytest.raises(ValueError, match="v: expected"):
            fa.cache_append(cache, new, new, table, zero)
        v.set_(old["v"].clone())
    assert torch.equal(fa.cache_fwd(q, cache, table, ln)[0], want)
    fa.sync_status()


# ------------------------------------------------------------------ eviction
@pytest.mark.parametrize("d,page,budget", [(64, 16, 20), (64, 64, 1)])
def test_evict_lengths_in_place(d, page, budget):
    """new_lens may be lens itself, with more heads than the GPU works on at
    once: every head is cut back from the old length."""
    import ctypes
    import struct
    fa = require_gpu()
    H, B, recent = 700, 2, 1
    lens = [100, 37]
    cache, table, ln = R.make(fa, lens, H, d, page, seed=38, spare=2 * (-(-budget // page)))
    used = set(table.flatten().tolist())
    per = -(-budget // page)
    dst = torch.tensor([p for p in range(cache.num_pages) if p not in used][:B * per], dtype=torch.int32).view(B, per).cuda()
    w = torch.rand(B, H, table.shape[1] * page, generator=torch.Generator().manual_seed(39)).cuda()
    want_lens, want_kept, want_w = fa.cache_evict(cache, table, ln, w, dst, budget, recent)
    fa.sync_status()
    kept, out = torch.full_like(want_kept, -7), torch.full_like(want_w, -7)
    c = struct.pack("@5P4i", *(t.data_ptr() for t in (cache.k, cache.v, cache.ks, cache.vs, cache.kb)), cache.num_pages, H,
                    page, d)
    lib = fa.load_library()
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    call = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_char_p, *[ctypes.c_void_p] * 4, *[ctypes.c_int] * 5,
                            *[ctypes.c_void_p] * 4)(("fa4fp4_cache_evict", lib))
    in_place = ln.clone()
    torch.cuda.synchronize()
    assert call(c, p(table), p(in_place), p(w), p(dst), B, table.shape[1], per, budget, recent, p(in_place), p(kept), p(out),
                ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    fa.sync_status()
    assert torch.equal(in_place, want_lens) and torch.equal(kept, want_kept) and torch.equal(out, want_w)


# ------------------------------------------------------------------ what else the calls allow
def fa_values(cache):
    """|v| of every finite code in the pages, under their scales."""
    v = np.abs(np.nan_to_num(R.E4M3[cache.v.cpu().numpy()]))
    used = (cache.vs.cpu().numpy() != 200)[:, :, None, None]
    return np.where(used, v * 2.0 ** (cache.vs.cpu().numpy().astype(np.float64) - 127)[:, :, None, None], 0)


@pytest.mark.parametrize("f32", [True, False])
def test_pages_listed_twice(f32):
    """A page that is listed twice counts twice: o is the mean over the doubled
    keys, and lse of pages that are all listed twice is ln 2 higher."""
    fa = require_gpu()
    d, page, H, G, T = 64, 16, 2, 4, 2
    cache, table, ln = R.make(fa, [150, 70], H, d, page, seed=43)
    q = queries(2, H * G, T, d, 44)
    once = torch.tensor([0, 2, 3], dtype=torch.int32).expand(2, H, T, 3).contiguous().cuda()
    twice = torch.tensor([2, 0, 3, 3, 2, 0], dtype=torch.int32).expand(2, H, T, 6).contiguous().cuda()
    mixed = torch.tensor([3, 0, 3, 2, -1], dtype=torch.int32).expand(2, H, T, 5).contiguous().cuda()
    dt = fa.OUT_F32 if f32 else fa.OUT_BF16
    o1, l1 = fa.cache_fwd(q, cache, table, ln, pages=once, out_dtype=dt)
    o2, l2 = fa.cache_fwd(q, cache, table, ln, pages=twice, out_dtype=dt)
    fa.sync_status()
    # The scores are the same.  Each side's weights carry the exponential (2^-19 of the
    # spread) and P's f16 (2^-22 or 2^-11), each output half a step; |v| < 8
    assert float(fa_values(cache).max()) < 8
    tol = 2 * 8 * (2.0 ** -19 + (2.0 ** -22 + 2.0 ** -24 if f32 else 2.0 ** -11 + 2.0 ** -8))
    assert np.abs(f64(o1) - f64(o2)).max() <= tol and np.abs(f64(l2) - f64(l1) - np.log(2)).max() <= 2 * 2.0 ** -18
    check(fa, q, cache, table, ln, [150, 70], f32, pages=mixed)


@pytest.mark.parametrize("B,H", [(100, 1), (300, 2)])
@pytest.mark.parametrize("G,T", [(4, 1), (2, 7)])
def test_many_sequences_few_rows(B, H, G, T):
    """More sequences than a warp has lanes, few enough to be cut at their ends and
    too many for that: attention, received weights and selection, with lengths of
    zero in runs, queries that are none, and room in the table."""
    fa = require_gpu()
    d, page = 64, 32
    g = torch.Generator().manual_seed(45)
    lens = torch.randint(0, 700, (B,), generator=g)
    lens[10:60] = 0
    lens[70:90] = torch.arange(20)
    q_lens = torch.randint(0, T + 1, (B,), generator=g)
    cache, table, ln = R.make(fa, lens.tolist(), H, d, page, seed=46, room=500)
    q = queries(B, H * G, T, d, 47)
    ql = q_lens.int().cuda()
    o = torch.full(q.shape, 7.0, device="cuda")
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    fa.cache_fwd(q, cache, table, ln, q_lens=ql, out=o, lse=lse, out_dtype=fa.OUT_F32)
    w = torch.rand(B, H, table.shape[1] * page, device="cuda")
    got = fa.cache_weigh(q, lse, cache, table, ln, w, q_lens=ql, out=torch.full_like(w, 5.0))
    sel = fa.cache_select(q, cache, table, ln, 4, q_lens=ql)
    fa.sync_status()
    ref = R.Ref.of(cache, table)
    wo, wl, spread, eps, small = ref.fwd(f64(q), lens, q_lens)
    e = eps * d * 2.0 ** -23
    rows = np.broadcast_to(np.arange(T)[None, None] < q_lens.numpy()[:, None, None], wl.shape)
    tol = (4 * e + 2.0 ** -19 + 2.0 ** -22)[..., None] * spread + 2.0 ** -24 * np.abs(wo) + small[..., None]
    assert (np.abs(f64(o) - wo) <= tol)[rows].all() and (f64(o)[~rows] == 7).all() and (f64(lse)[~rows] == 7).all()
    assert np.array_equal(np.isneginf(f64(lse))[rows], np.isneginf(wl)[rows])
    assert np.array_equal(sel.cpu().numpy(), ref.select(f64(q), lens, q_lens, 4))
    want = ref.weigh(f64(q), np.where(rows, f64(lse), -np.inf), lens, q_lens, f64(w))
    for b, n in enumerate(lens.tolist()):
        recv = want[b, :, :n] - f64(w)[b, :, :n]
        # as in the weights' own test: 2^-16 + 2^-21 |lse| with |lse| <= 16
        tol = (2 * e[b].max(initial=0) + 2.0 ** -15) * recv + 2.0 ** -22 * want[b, :, :n]
        assert (np.abs(f64(got[b, :, :n]) - want[b, :, :n]) <= tol).all() and (got[b, :, n:] == 5).all()


def test_full_cache_and_no_new_tokens():
    """Sequences at the table's capacity: nothing to append is no error."""
    fa = require_gpu()
    d, page, H = 64, 16, 2
    cache, table, ln = R.make(fa, [48, 48, 20], H, d, page, seed=48)
    before = [t.clone() for t in (cache.k, cache.v, cache.ks, cache.vs, cache.kb)]
    x = queries(3, H, 5, d, 49)
    fa.cache_append(cache, x, x, table, ln, n_new=torch.zeros(3, dtype=torch.int32, device="cuda"))
    fa.sync_status()
    for a, b in zip(before, (cache.k, cache.v, cache.ks, cache.vs, cache.kb)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("G,T", [(4, 1), (4, 30)])
def test_padded_rows_hold_anything(G, T):
    """NaN and infinities in query rows behind q_lens and in their lse reach
    nothing."""
    fa = require_gpu()
    d, page, H = 128, 64, 2
    lens, q_lens = [200, 90, 131], [T, 0, (T + 1) // 2]
    cache, table, ln = R.make(fa, lens, H, d, page, seed=50)
    ql = torch.tensor(q_lens, dtype=torch.int32).cuda()
    q = queries(3, H * G, T, d, 51)
    bad = q.clone()
    for b, n in enumerate(q_lens):
        bad[b, :, n:] = float("nan") if b else float("inf")
    w = torch.rand(3, H, table.shape[1] * page, device="cuda")
    for f32 in (False, True):
        dt = fa.OUT_F32 if f32 else fa.OUT_BF16
        o1, l1 = fa.cache_fwd(q, cache, table, ln, q_lens=ql, out_dtype=dt)
        o2, l2 = fa.cache_fwd(bad, cache, table, ln, q_lens=ql, out_dtype=dt)
        assert torch.equal(o1, o2) and torch.equal(l1, l2)
    nan = l1.clone()
    for b, n in enumerate(q_lens):
        nan[b, :, n:] = float("nan")
    a = fa.cache_weigh(q, l1, cache, table, ln, w, q_lens=ql, out=w.clone())
    b = fa.cache_weigh(bad, nan, cache, table, ln, w, q_lens=ql, out=w.clone())
    assert torch.equal(a, b)
    assert torch.equal(fa.cache_select(q, cache, table, ln, 2, q_lens=ql), fa.cache_select(bad, cache, table, ln, 2, q_lens=ql))
    fa.sync_status()


@pytest.mark.parametrize("d,page,H,G,T,f32", FEW)
def test_fwd_small_queries(d, page, H, G, T, f32):
    """As in the kernel for many rows: query rows down to the smallest bf16 over pages
    of zero keys and of very small ones, with pool page 0 unused."""
    fa = require_gpu()
    g = torch.Generator().manual_seed(52)
    lens = [T + 5, 300, 128, 7, 290]
    k = [torch.randn(H, n, d, generator=g) for n in lens]
    k[1][:, 100:] = 0
    k[2][:, 60:] *= 2.0 ** -120
    k[4][:] = 0
    v = [torch.randn(H, n, d, generator=g) for n in lens]
    cache, table, ln, lens = cache_of(fa, k, v, page, 53, first=1)
    q = queries(len(lens), H * G, T, d, 54)
    q *= (2.0 ** -(torch.arange(H * G) % 14 * 10).float()).view(1, H * G, 1, 1).cuda()
    for causal in (True, False):
        for scale in (None, 1e-12):
            check(fa, q, cache, table, ln, lens, f32, causal, scale)


# ------------------------------------------------------------------ keys and queries far apart
def around_one(*shape, seed):
    """Magnitudes in [0.5, 2): exact under any power of two that bf16 has."""
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(*shape, generator=g) * 1.5 + 0.5).bfloat16().float() * (torch.randint(0, 2, shape, generator=g) * 2 - 1)


@pytest.mark.parametrize("k_up,q_up", [(120, -112), (-112, 120)])
@pytest.mark.parametrize("d,page,H,G,T,f32", FEW + [(128, 64, 1, 2, 70, False), (64, 16, 1, 3, 90, True)])
def test_fwd_keys_and_queries_far_apart(d, page, H, G, T, f32, k_up, q_up):
    """Keys near one end of bf16's range under queries near the other, of scores of
    ordinary size."""
    fa = require_gpu()
    lens = [T, 150, 700]
    k = [around_one(H, n, d, seed=55 + i) * 2.0 ** k_up for i, n in enumerate(lens)]
    v = [around_one(H, n, d, seed=60 + i) for i, n in enumerate(lens)]
    cache, table, ln, lens = cache_of(fa, k, v, page, 56)
    q = (around_one(len(lens), H * G, T, d, seed=57) * 2.0 ** q_up).bfloat16().cuda()
    check(fa, q, cache, table, ln, lens, f32, scale=2.0 ** -7)


@pytest.mark.parametrize("k_up,q_up", [(120, -112), (-112, 120)])
@pytest.mark.parametrize("d,page,G,T", WEIGH)
def test_weigh_keys_and_queries_far_apart(d, page, G, T, k_up, q_up):
    """The same weights, bit for bit, as under keys and queries of ordinary size, whose
    scores differ by nothing but powers of two that cancel."""
    fa = require_gpu()
    H, lens = 2, [T + 150, T, 129]
    k = [around_one(H, n, d, seed=58 + i) for i, n in enumerate(lens)]
    q = around_one(3, H * G, T, d, seed=59)
    got = []
    for ku, qu in ((k_up + q_up, 0), (k_up, q_up)):
        cache, table, ln, _ = cache_of(fa, [x * 2.0 ** ku for x in k], k, page, 60)
        x, scale = (q * 2.0 ** qu).bfloat16().cuda(), 0.03
        w = torch.zeros(3, H, table.shape[1] * page, device="cuda")
        if not got:
            _, lse = fa.cache_fwd(x, cache, table, ln, softmax_scale=scale, out_dtype=fa.OUT_F32)
        got.append(fa.cache_weigh(x, lse, cache, table, ln, w, softmax_scale=scale))
    fa.sync_status()
    assert torch.equal(*got)
