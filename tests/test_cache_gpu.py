"""The 8-bit cache on the GPU against the plain 64-bit reference (cache_ref.py).

Codes, scales, bounds, selected pages and kept positions are compared exactly.

Attention: with eps = 2^-23 * d * max_j scale * sum |q| |k_j| the error of a
score (FP32 sum of d exact products, one step of 2^-23 each, whatever their
order) every weight is off by at most 2 eps + 2^-20 relative (the exponential,
its argument and the running rescales), and P itself by 2^-11 (f16 has 11
significant bits: steps of 2^-10 in [1, 2) * 2^k, so half a step is up to 2^-11
of the value) or 2^-22 (the sum of two f16).  Numerator
and normalizer each carry the weights' error, so
  |o - ref| <= (4 eps + 2^-19 + p_err) * spread + out_err * |ref| + 2^-35 n V,
with n keys and V their largest |v|: P times 2^15 times the ratio of V's page
scale to the accumulator's (at most 2^4 above the largest of the keys that are
multiplied together) is a f16 number, whose smallest step is 2^-24; half of it
is 2^-25 2^-15 2^4 = 2^-36 of a scale 2^X with 448 * 2^X < 2 V, and the weights'
sum is at least 1.  (The kernel for many rows: 2^12 and at most 2^1, the same.)
spread = sum p |v| / sum p, and out_err half a step of the output's type: 2^-8
bf16, 2^-24 FP32.
  |lse - ref| <= 2 eps + 2^-20 + 2^-22 |ref|."""
import numpy as np
import pytest
import torch

import cache_ref as R
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def check_fwd(o, lse, ref, d, f32, rows=None):
    ro, rl, spread, eps, small = ref
    e = eps * d * 2.0 ** -23
    tol = (4 * e + 2.0 ** -19 + (2.0 ** -22 if f32 else 2.0 ** -11))[..., None] * spread
    tol += (2.0 ** -24 if f32 else 2.0 ** -8) * np.abs(ro) + small[..., None] + 1e-37
    o, lse = f64(o), f64(lse)
    rows = np.ones(rl.shape, bool) if rows is None else rows
    assert np.isfinite(o[rows]).all()
    bad = np.abs(o - ro)[rows] - tol[rows]
    assert bad.max(initial=-1) <= 0, f"o off by {bad.max():.3g} over its bound"
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse)[rows], empty[rows])
    assert not o[rows & empty].any()
    sel = rows & ~empty
    lt = 2 * e + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(empty, 0, rl))
    assert (np.abs(lse[sel] - rl[sel]) <= lt[sel]).all()


def queries(B, Hq, T, d, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, Hq, T, d, generator=g) * scale).to(torch.bfloat16).cuda()


def same_contents(cache, ref):
    for got, want in zip(R.contents(cache), [R.E4M3[ref.k], R.E4M3[ref.v], R.E4M3[ref.kb], ref.ks, ref.vs]):
        assert np.array_equal(got, want, equal_nan=got.dtype.kind == "f")


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append(d, page):
    """Several appends of every length onto partly filled pages, magnitudes
    rising and falling so that some raise a page's exponent."""
    fa = require_gpu()
    B, H, room = 5, 3, 3 * page + 40
    cache, table, _ = R.make(fa, [0] * B, H, d, page, seed=d + page, room=room)
    ref = R.Ref.of(cache, table)
    lens = np.zeros(B, dtype=np.int64)
    g = torch.Generator().manual_seed(page)
    for step, (T, mag) in enumerate([(1, 1.0), (page - 1, 0.01), (1, 300.0), (page + 5, 1e-6), (2, 1e6), (33, 1.0)]):
        k = (torch.randn(B, H, T, d, generator=g) * mag).to(torch.bfloat16)
        v = (torch.randn(B, H, T, d, generator=g) * mag ** 0.5).to(torch.bfloat16)
        if step == 1:
            k[0] = 0
            v[1, :, :, 1:] = 0
        n = torch.randint(0, T + 1, (B,), generator=g).numpy() if step >= 3 else np.full(B, T)
        fa.cache_append(cache, k.cuda(), v.cuda(), table, torch.tensor(lens, dtype=torch.int32).cuda(),
                        n_new=None if step < 3 else torch.tensor(n, dtype=torch.int32).cuda())
        ref.append(k.double().numpy(), v.double().numpy(), lens, n)
        lens += n
        same_contents(cache, ref)
    fa.sync_status()


def test_append_extreme_values():
    """The largest and smallest bf16 magnitudes, amax on the exponent rule's
    edges, and -0."""
    fa = require_gpu()
    d, page = 64, 16
    edge = [448.0, 450.0, 446.0, 512.0, 0.875, 0.8789, 2.0 ** -126, 2.0 ** -133, 3.3895e38, -3.3895e38, 1e-38, -0.0]
    cache, table, _ = R.make(fa, [0] * len(edge), 1, d, page, room=page)
    ref = R.Ref.of(cache, table)
    k = torch.zeros(len(edge), 1, 3, d)
    for i, x in enumerate(edge):
        k[i, 0, 0, 5] = x
        k[i, 0, 1] = torch.linspace(-1, 1, d) * abs(x)
        k[i, 0, 2] = torch.logspace(-8, 0, d) * x
    k = k.to(torch.bfloat16)
    lens = np.zeros(len(edge), dtype=np.int64)
    fa.cache_append(cache, k.cuda(), (-k).cuda(), table, torch.tensor(lens, dtype=torch.int32).cuda())
    ref.append(k.double().numpy(), -k.double().numpy(), lens, np.full(len(edge), 3))
    same_contents(cache, ref)
    fa.sync_status()


def test_append_nonfinite_is_flagged_and_stored_finite():
    fa = require_gpu()
    d, page = 64, 16
    cache, table, _ = R.make(fa, [0, 0], 2, d, page, room=page)
    fa.sync_status()
    ref = R.Ref.of(cache, table)
    x = torch.randn(2, 2, 4, d).to(torch.bfloat16)
    y = x.clone()
    x[0, 1, 2, 3], x[0, 1, 1, 4], x[1, 0, 0, 0] = float("nan"), float("-inf"), float("inf")
    y[0, 1, 2, 3] = 0
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    fa.cache_append(cache, x.cuda(), y.cuda(), table, zero)
    with pytest.raises(fa.Fa4Fp4Error) as e:
        fa.sync_status()
    assert e.value.status == 8
    fa.sync_status()
    # the infinities saturate without a say in the exponent
    z = y.double().numpy()
    z[0, 1, 1, 4], z[1, 0, 0, 0] = 0, 0
    ref.append(z, y.double().numpy(), np.zeros(2, int), np.full(2, 4))
    got = R.contents(cache)
    assert np.array_equal(got[3], ref.ks) and np.array_equal(got[4], ref.vs)
    tb = table.cpu().numpy()
    assert got[0][tb[0, 0], 1, 1, 4] == -448 and got[0][tb[1, 0], 0, 0, 0] == 448 and got[0][tb[0, 0], 1, 2, 3] == 0


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,page,H,G,T", [(64, 16, 2, 1, 1), (64, 64, 1, 4, 3), (64, 128, 2, 5, 1), (64, 32, 3, 3, 6),
                                          (128, 16, 1, 8, 2), (128, 32, 2, 7, 1), (128, 64, 2, 4, 1),
                                          (128, 128, 1, 2, 17), (128, 64, 1, 16, 1), (128, 16, 2, 12, 1)])
def test_fwd(d, page, H, G, T, causal, f32):
    """Lengths on and around every boundary, none at all, rows that see
    nothing, ragged query counts; NaN codes behind every end."""
    fa = require_gpu()
    lens = [0, 1, 2, page - 1, page, page + 1, 31, 127, 128, 129, 300]
    q_lens = [0, 1, T, T, 1, T, (T + 1) // 2, T, T, 0, T]
    if T > 2:
        q_lens[2] = T                 # more queries than tokens: the first see nothing
    cache, table, ln = R.make(fa, lens, H, d, page, seed=1)
    q = queries(len(lens), H * G, T, d, 2)
    ql = torch.tensor(q_lens, dtype=torch.int32).cuda()
    dt = fa.OUT_F32 if f32 else fa.OUT_BF16
    o = torch.full(q.shape, 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    fa.cache_fwd(q, cache, table, ln, q_lens=ql, causal=causal, out_dtype=dt, out=o, lse=lse)
    rows = np.arange(T)[None, None, :] < np.array(q_lens)[:, None, None]
    rows = np.broadcast_to(rows, lse.shape)
    check_fwd(o, lse, R.Ref.of(cache, table).fwd(f64(q), lens, q_lens, causal), d, f32, rows)
    assert (f64(o)[~rows] == 7).all() and (f64(lse)[~rows] == 7).all()
    o2, l2 = fa.cache_fwd(q, cache, table, ln, q_lens=ql, causal=causal, out_dtype=dt)
    assert torch.equal(o2.cpu()[torch.tensor(rows)], o.cpu()[torch.tensor(rows)])
    o3, l3 = fa.cache_fwd(q, cache, table, ln, q_lens=ql, causal=causal, out_dtype=dt, with_lse=False)
    assert l3 is None and torch.equal(o3, o2)
    fa.sync_status()


@pytest.mark.parametrize("lens,G,T", [([20001], 4, 1), ([1, 9000, 3, 2500], 8, 1), ([5000, 700], 4, 4),
                                      ([2047] * 9, 1, 1)])
@pytest.mark.parametrize("d,page", [(128, 64), (64, 16)])
def test_fwd_split(lens, G, T, d, page):
    """Few rows over long caches: the keys are split over the GPU and joined."""
    fa = require_gpu()
    H = 2
    cache, table, ln = R.make(fa, lens, H, d, page, seed=3)
    q = queries(len(lens), H * G, T, d, 4, scale=2.0)
    o, lse = fa.cache_fwd(q, cache, table, ln, out_dtype=fa.OUT_F32)
    ql = [T] * len(lens)
    check_fwd(o, lse, R.Ref.of(cache, table).fwd(f64(q), lens, ql), d, True)
    ob, _ = fa.cache_fwd(q, cache, table, ln)
    check_fwd(ob, lse, R.Ref.of(cache, table).fwd(f64(q), lens, ql), d, False)
    fa.sync_status()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,page,H,G,T", [(128, 64, 8, 4, 70), (128, 16, 8, 1, 300), (64, 128, 8, 5, 60), (64, 32, 16, 2, 129),
                                          (128, 32, 8, 16, 20), (128, 128, 8, 3, 100)])
def test_fwd_chunk(d, page, H, G, T, causal):
    """Many query tokens per sequence and enough heads for the kernel that takes
    256 rows at a time; contexts shorter than the chunk, none at all, ragged
    query counts, NaN codes behind every end."""
    fa = require_gpu()
    lens = [T + 150, T, 0, T // 2, 515, T + 128 - T % 128]
    q_lens = [T, T, T, T, T - 1, 3]
    cache, table, ln = R.make(fa, lens, H, d, page, seed=40)
    q = queries(len(lens), H * G, T, d, 41)
    ql = torch.tensor(q_lens, dtype=torch.int32).cuda()
    o = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    fa.cache_fwd(q, cache, table, ln, q_lens=ql, causal=causal, out=o, lse=lse)
    fa.sync_status()
    rows = np.broadcast_to(np.arange(T)[None, None, :] < np.array(q_lens)[:, None, None], lse.shape)
    check_fwd(o, lse, R.Ref.of(cache, table).fwd(f64(q), lens, q_lens, causal), d, False, rows)
    assert (f64(o)[~rows] == 7).all() and (f64(lse)[~rows] == 7).all()
    o2, l2 = fa.cache_fwd(q, cache, table, ln, q_lens=ql, causal=causal, with_lse=False)
    assert l2 is None and torch.equal(o2.cpu()[torch.tensor(rows)], o.cpu()[torch.tensor(rows)])


def test_fwd_chunk_scales_far_apart():
    """As below, through the kernel for many rows: pages whose V scales differ
    by up to 2^77 and K scales by 4."""
    fa = require_gpu()
    d, page, H, G, T = 128, 16, 8, 4, 128
    lens = [300, 300, 41]
    cache, table, ln = R.make(fa, lens, H, d, page, seed=42)
    g = torch.Generator().manual_seed(43)
    k = torch.randn(3, H, 300, d, generator=g)
    v = torch.randn(3, H, 300, d, generator=g)
    for i in range(0, 300, page):
        v[:, :, i:i + page] *= 2.0 ** (40 - 7 * (i // page % 12))
        k[:, :, i:i + page] *= 2.0 ** (i // page % 3)
    fa.cache_append(cache, k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), table, torch.zeros_like(ln), n_new=ln)
    q = queries(3, H * G, T, d, 44)
    q[0, 5] *= 1e-20
    q[1, 7] = 0
    q[2, 9, 100, 3] = float("nan")
    o, lse = fa.cache_fwd(q, cache, table, ln, softmax_scale=0.2)
    fa.sync_status()
    rows = np.ones(lse.shape, bool)
    rows[2, 9, 100] = False
    check_fwd(o, lse, R.Ref.of(cache, table).fwd(np.nan_to_num(f64(q)), lens, [T] * 3, scale=0.2), d, False, rows)
    assert torch.isnan(o[2, 9, 100]).all()


@pytest.mark.parametrize("d,page,H,G,T,causal", [(128, 64, 2, 4, 40, True), (64, 16, 1, 2, 150, False),
                                                 (128, 128, 1, 16, 33, True), (64, 32, 2, 3, 60, True)])
def test_fwd_chunk_cut(d, page, H, G, T, causal):
    """Few blocks of rows and long contexts, so that a block's keys are cut among
    many CTAs; a workspace of other bytes, used again by another call between."""
    fa = require_gpu()
    lens = [4000, T, 2049, 0, 8191]
    q_lens = [T, T, T - 1, T, T]
    B = len(lens)
    cache, table, ln = R.make(fa, lens, H, d, page, seed=70)
    q = queries(B, H * G, T, d, 71)
    ql = torch.tensor(q_lens, dtype=torch.int32).cuda()
    ref = R.Ref.of(cache, table).fwd(f64(q), lens, q_lens, causal)
    rows = np.broadcast_to(np.arange(T)[None, None, :] < np.array(q_lens)[:, None, None], ref[1].shape)
    need = fa.cache_fwd_workspace_bytes(B, H * G, H, T, d, page, table.shape[1])
    ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
    got = []
    for i in range(3):
        o, lse = fa.cache_fwd(q, cache, table, ln, q_lens=ql, causal=causal, workspace=ws)
        got.append(o.clone())
        check_fwd(o, lse, ref, d, False, rows)
        # the same workspace, other uses of it: the counter words are left ready
        few = fa.cache_fwd(q[:, :, :1].contiguous(), cache, table, ln, workspace=ws)[0]
        if i:
            assert torch.equal(few, last)
        last = few
    sel = torch.tensor(np.ascontiguousarray(rows))
    assert torch.equal(got[0].cpu()[sel], got[1].cpu()[sel]) and torch.equal(got[0].cpu()[sel], got[2].cpu()[sel])
    with pytest.raises(fa.Fa4Fp4Error) as e:
        fa.cache_fwd(q, cache, table, ln, q_lens=ql, causal=causal, workspace=ws[: need - 1])
    assert e.value.status == 6
    fa.sync_status()


@pytest.mark.parametrize("causal", [True, False])
def test_fwd_chunk_many_sequences(causal):
    """More sequences and blocks of rows than a warp looks up at once, with and
    without queries, shorter and longer than their queries."""
    fa = require_gpu()
    d, page, H, G, T, B = 64, 32, 2, 8, 40, 150
    g = torch.Generator().manual_seed(72)
    lens = torch.randint(0, 300, (B,), generator=g).tolist()
    q_lens = torch.randint(0, T + 1, (B,), generator=g).tolist()
    q_lens[40:110] = [0] * 70
    lens[45] = 0
    cache, table, ln = R.make(fa, lens, H, d, page, seed=73)
    q = queries(B, H * G, T, d, 74)
    ql = torch.tensor(q_lens, dtype=torch.int32).cuda()
    o = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    fa.cache_fwd(q, cache, table, ln, q_lens=ql, causal=causal, out=o, lse=lse)
    fa.sync_status()
    rows = np.broadcast_to(np.arange(T)[None, None, :] < np.array(q_lens)[:, None, None], lse.shape)
    check_fwd(o, lse, R.Ref.of(cache, table).fwd(f64(q), lens, q_lens, causal), d, False, rows)
    assert (f64(o)[~rows] == 7).all() and (f64(lse)[~rows] == 7).all()


def test_fwd_chunk_bad_page():
    fa = require_gpu()
    d, page, H, G, T = 64, 32, 8, 4, 100
    lens = [200, 300, 250]
    cache, table, ln = R.make(fa, lens, H, d, page, seed=45)
    q = queries(3, H * G, T, d, 46)
    want = R.Ref.of(cache, table).fwd(f64(q), lens, [T] * 3)
    t = table.clone()
    t[1, 4] = cache.num_pages
    o, lse = fa.cache_fwd(q, cache, t, ln)
    with pytest.raises(fa.Fa4Fp4Error) as e:
        fa.sync_status()
    assert e.value.status == 7
    rows = np.ones(lse.shape, bool)
    rows[1] = False
    check_fwd(o, lse, want, d, False, rows)
    assert np.isfinite(f64(o)).all()


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("T", [1, 3, 60])
def test_fwd_large_scores(T, f32):
    """Scores that are multiples of 2^19, up to 7 * 2^19: of a row's keys only
    those with the largest count, all alike.  Their weights are 2^x with the same
    x, which the rounding of the reference (at most 2^-2 at 2^22) leaves within
    the range of P: the mean of their values, to the roundings of P (2^-11 or
    2^-22, the same for all), of the sums and of the output."""
    fa = require_gpu()
    d, page, H, G, n = 128, 16, 1, 4, 600
    cache, table, ln = R.make(fa, [n], H, d, page, seed=75)
    g = torch.Generator().manual_seed(76)
    j = torch.randint(0, 8, (n,), generator=g)
    v = torch.randint(-8, 9, (1, H, n, d), generator=g)
    k = (j.view(1, 1, n, 1) * torch.ones(1, H, n, d)).bfloat16().cuda()
    fa.cache_append(cache, k, v.bfloat16().cuda(), table, torch.zeros_like(ln), n_new=ln)
    q = torch.full((1, H * G, T, d), 4096.0).bfloat16().cuda()
    o, lse = fa.cache_fwd(q, cache, table, ln, softmax_scale=1.0, out_dtype=fa.OUT_F32 if f32 else fa.OUT_BF16)
    fa.sync_status()
    o, lse = f64(o), f64(lse)
    for t in range(T):
        see = n - T + t + 1
        top = (j[:see] == j[:see].max()).numpy()
        want = v[0, 0, :see].numpy()[top].mean(0)
        tol = (2.0 ** -10 if not f32 else 2.0 ** -16) * np.abs(v[0, 0, :see].numpy()[top]).mean(0)
        tol = tol + (2.0 ** -24 if f32 else 2.0 ** -8) * np.abs(want)
        assert (np.abs(o[0, :, t] - want) <= tol).all()
        # a unit in the last place of 2^22 is 2^-1: the roundings of log2 e, of the
        # score in log2 units, of ln 2 and of the result are half of one each
        assert (np.abs(lse[0, :, t] - int(j[:see].max()) * 2.0 ** 19 - np.log(top.sum())) <= 2.0).all()


@pytest.mark.parametrize("T", [1, 40, 200])
def test_fwd_scales_far_apart(T):
    """Pages whose scales differ by 2^40, keys of a magnitude that leaves one
    of them with all the weight, and an explicit softmax scale."""
    fa = require_gpu()
    d, page, H, G = 128, 16, 1, 4
    lens = [200]
    cache, table, ln = R.make(fa, lens, H, d, page, seed=5)
    g = torch.Generator().manual_seed(6)
    k = torch.randn(1, H, 200, d, generator=g)
    v = torch.randn(1, H, 200, d, generator=g)
    for i in range(0, 200, page):
        v[:, :, i:i + page] *= 2.0 ** (40 - 7 * (i // page % 12))
        k[:, :, i:i + page] *= 2.0 ** (i // page % 3)
    fa.cache_append(cache, k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), table, torch.zeros_like(ln))
    q = queries(1, H * G, T, d, 7)
    for f32 in (True, False):
        o, lse = fa.cache_fwd(q, cache, table, ln, softmax_scale=0.2, out_dtype=fa.OUT_F32 if f32 else fa.OUT_BF16)
        ref = R.Ref.of(cache, table).fwd(f64(q), lens, [T], scale=0.2)
        check_fwd(o, lse, ref, d, f32)
    fa.sync_status()


def test_fwd_query_magnitudes():
    """Query rows of very different magnitude, zeros, and a row with a NaN:
    the others of its block are not touched by it."""
    fa = require_gpu()
    d, page, H, G = 64, 32, 1, 8
    lens = [150]
    cache, table, ln = R.make(fa, lens, H, d, page, seed=8)
    q = queries(1, H * G, 1, d, 9)
    for h, s in enumerate([1e-30, 1e-6, 1.0, 30.0, 0.0, 1e-3, 4.0, 1.0]):
        q[0, h] *= s
    o, lse = fa.cache_fwd(q, cache, table, ln, out_dtype=fa.OUT_F32)
    check_fwd(o, lse, R.Ref.of(cache, table).fwd(f64(q), lens, [1]), d, True)
    bad = q.clone()
    bad[0, 3, 0, 5] = float("nan")
    o2, _ = fa.cache_fwd(bad, cache, table, ln, out_dtype=fa.OUT_F32)
    keep = [h for h in range(8) if h != 3]
    assert torch.equal(o2[0, keep], o[0, keep]) and torch.isnan(o2[0, 3]).all()
    fa.sync_status()


def test_fwd_offsets_past_32_bits():
    """Pages more than 2^32 bytes into the pool."""
    fa = require_gpu()
    d, page, H, G = 128, 128, 8, 2
    first = (1 << 32) // (H * page * d) + 5
    lens = [300, 129]
    cache, table, ln = R.make(fa, lens, H, d, page, seed=10, first=first)
    assert int(table.min()) * H * page * d > 1 << 32
    base = int(table.min())
    small = R.Ref(*(t[base:].cpu().numpy() for t in (cache.k, cache.v, cache.ks, cache.vs, cache.kb)),
                  (table - base).cpu().numpy())
    q = queries(2, H * G, 2, d, 11)
    o, lse = fa.cache_fwd(q, cache, table, ln, out_dtype=fa.OUT_F32)
    check_fwd(o, lse, small.fwd(f64(q), lens, [2, 2]), d, True)
    sel = fa.cache_select(q, cache, table, ln, 2)
    assert np.array_equal(sel.cpu().numpy(), small.select(f64(q), lens, [2, 2], 2))
    fa.sync_status()


# ------------------------------------------------------------------ sparse
@pytest.mark.parametrize("d,page,H,G,T,n_sel", [(64, 16, 2, 1, 1, 1), (64, 16, 2, 3, 3, 4), (128, 64, 2, 4, 1, 3),
                                                (128, 32, 1, 8, 2, 200), (128, 16, 1, 20, 1, 7), (64, 128, 2, 2, 5, 2)])
def test_select_and_sparse_fwd(d, page, H, G, T, n_sel):
    fa = require_gpu()
    lens = [0, 1, page, page + 1, 5 * page + 3, 20 * page, 33 * page - 1, 150]
    q_lens = [T, 1, T, T, T, 0, T, (T + 1) // 2]
    cache, table, ln = R.make(fa, lens, H, d, page, seed=12)
    q = queries(len(lens), H * G, T, d, 13)
    ql = torch.tensor(q_lens, dtype=torch.int32).cuda()
    ref = R.Ref.of(cache, table)
    sel = fa.cache_select(q, cache, table, ln, n_sel, q_lens=ql)
    want = ref.select(f64(q), lens, q_lens, n_sel)
    assert np.array_equal(sel.cpu().numpy(), want)
    rows = np.broadcast_to(np.arange(T)[None, None] < np.array(q_lens)[:, None, None], (len(lens), H * G, T))
    for f32 in (False, True):
        o, lse = fa.cache_fwd(q, cache, table, ln, q_lens=ql, pages=sel, out_dtype=fa.OUT_F32 if f32 else fa.OUT_BF16)
        check_fwd(o, lse, ref.fwd(f64(q), lens, q_lens, pages=want), d, f32, rows)
    # lists in another order, and with holes
    perm = torch.randperm(n_sel, generator=torch.Generator().manual_seed(1))
    o2, l2 = fa.cache_fwd(q, cache, table, ln, q_lens=ql, pages=sel[..., perm.cuda()].contiguous(), out_dtype=fa.OUT_F32)
    check_fwd(o2, l2, ref.fwd(f64(q), lens, q_lens, pages=want), d, True, rows)
    fa.sync_status()


@pytest.mark.parametrize("n_pages,n_sel", [(40, 9), (600, 300), (2000, 64), (16390, 5000)])
def test_select_ties(n_pages, n_sel):
    """Equal pages tie to the lowest; hundreds of them are all undecided in
    FP32."""
    fa = require_gpu()
    d, page, H = 64, 16, 1
    lens = [n_pages * page]
    cache, table, ln = R.make(fa, lens, H, d, page, seed=14)
    k = torch.randn(1, H, page, d).to(torch.bfloat16)
    k = k.repeat(1, 1, n_pages, 1)
    k[0, 0, 7 * page:9 * page] *= 1.5                       # two pages above the rest
    k[0, 0, 20 * page:21 * page] *= 0.5
    fa.cache_append(cache, k.cuda(), k.cuda(), table, torch.zeros_like(ln))
    q = queries(1, 3, 1, d, 15)
    sel = fa.cache_select(q, cache, table, ln, n_sel).cpu().numpy()
    assert np.array_equal(sel, R.Ref.of(cache, table).select(f64(q), lens, [1], n_sel))
    fa.sync_status()


def test_select_near_ties():
    """Bounds that differ by less than FP32 can tell: one key element of each
    page, 2^-26 of the sum."""
    fa = require_gpu()
    d, page, n_pages = 128, 16, 64
    lens = [n_pages * page]
    cache, table, ln = R.make(fa, lens, 1, d, page, seed=16)
    g = torch.Generator().manual_seed(17)
    k = torch.randn(1, 1, page, d, generator=g).to(torch.bfloat16).repeat(1, 1, n_pages, 1)
    small = torch.randperm(n_pages, generator=g)
    for i in range(n_pages):
        k[0, 0, i * page:(i + 1) * page, 77] = (int(small[i]) - 32) / 32
    fa.cache_append(cache, k.cuda(), k.cuda(), table, torch.zeros_like(ln))
    q = torch.ones(1, 1, 1, d, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0, 77] = 2.0 ** -22
    for n_sel in (1, 2, 17, 40, 63, 64):
        sel = fa.cache_select(q, cache, table, ln, n_sel).cpu().numpy()
        assert np.array_equal(sel, R.Ref.of(cache, table).select(f64(q), lens, [1], n_sel))
    fa.sync_status()


# ------------------------------------------------------------------ weights
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,page,H,G,T", [(64, 16, 2, 1, 1), (128, 64, 2, 4, 1), (128, 128, 1, 3, 7), (64, 32, 2, 5, 40),
                                          (128, 64, 1, 4, 100), (128, 16, 2, 1, 300), (64, 16, 1, 8, 15), (128, 64, 1, 1, 79), (64, 32, 1, 4, 20),
                                          (128, 32, 2, 2, 63), (128, 32, 1, 1, 128), (64, 128, 1, 2, 9)])
def test_weigh(d, page, H, G, T, causal):
    """|out - ref| <= (2 eps + 2^-19 + 2^-21 |lse|) * received + 2^-22 * ref:
    a weight's exponent carries the score's error eps, the rounding of score
    and lse in log2 units, and the FP32 sum of at most 200 terms 2^-16 of what
    was received (2^-24 a term)."""
    fa = require_gpu()
    lens = [0, 1, page - 1, page + 1, 129, 260]
    q_lens = [T, 1, T, T, (T + 1) // 2, T]
    cache, table, ln = R.make(fa, lens, H, d, page, seed=18)
    q = queries(len(lens), H * G, T, d, 19)
    ql = torch.tensor(q_lens, dtype=torch.int32).cuda()
    _, lse = fa.cache_fwd(q, cache, table, ln, q_lens=ql, causal=causal, out_dtype=fa.OUT_F32)
    ref = R.Ref.of(cache, table)
    eps = ref.fwd(f64(q), lens, q_lens, causal)[3].max() * d * 2.0 ** -23
    w = torch.rand(len(lens), H, table.shape[1] * page, device="cuda")
    out = torch.full_like(w, 5.0)
    assert fa.cache_weigh(q, lse, cache, table, ln, w, q_lens=ql, causal=causal, out=out) is out
    z = f64(lse)
    want = ref.weigh(f64(q), z, lens, q_lens, f64(w), causal)
    got = f64(out)
    for b, n in enumerate(lens):
        assert (got[b, :, n:] == 5).all()
        recv = want[b, :, :n] - f64(w)[b, :, :n]
        top = np.abs(z[b][np.isfinite(z[b])]).max(initial=0)
        tol = (2 * eps + 2.0 ** -16 + 2.0 ** -21 * top) * recv + 2.0 ** -22 * want[b, :, :n]
        assert (np.abs(got[b, :, :n] - want[b, :, :n]) <= tol).all()
    # in place
    v = w.clone()
    fa.cache_weigh(q, lse, cache, table, ln, v, q_lens=ql, causal=causal)
    for b, n in enumerate(lens):
        assert torch.equal(v[b, :, :n], out[b, :, :n]) and torch.equal(v[b, :, n:], w[b, :, n:])
    fa.sync_status()


# ------------------------------------------------------------------ eviction
@pytest.mark.parametrize("d,page,budget,recent", [(64, 16, 40, 8), (128, 64, 64, 0), (128, 128, 130, 130), (64, 32, 1, 0),
                                                  (64, 32, 1, 1), (128, 16, 299, 17), (128, 64, 400, 5)])
@pytest.mark.parametrize("room", [0, 9000, 33000])
def test_evict(d, page, budget, recent, room):
    fa = require_gpu()
    H = 2
    lens = [0, 1, budget, budget + 1, 300, 2500]
    cache, table, ln = R.make(fa, lens, H, d, page, seed=20, spare=len(lens) * (-(-budget // page) + 1), room=room)
    # pages of very different scales meet in one destination page
    g = torch.Generator().manual_seed(21)
    x = torch.randn(1, H, 2500, d, generator=g) * 2.0 ** torch.randint(-12, 12, (1, 1, 2500, 1), generator=g).float()
    pad = torch.zeros(len(lens) - 1, H, 2500, d)
    n5 = torch.tensor([0, 0, 0, 0, 0, 2500], dtype=torch.int32).cuda()
    x = torch.cat([pad, x]).to(torch.bfloat16).cuda()
    fa.cache_append(cache, x, x, table, torch.zeros_like(ln), n_new=n5)
    used = set(table.flatten().tolist())
    free = torch.tensor([p for p in range(cache.num_pages) if p not in used], dtype=torch.int32)
    room = -(-budget // page) + 1
    dst = free[torch.randperm(len(free), generator=g)[:len(lens) * room]].view(len(lens), room).contiguous()
    w = torch.rand(len(lens), H, table.shape[1] * page, generator=g)
    w[4, :, 50:200] = 0.5                                  # ties
    w[5, 0, ::3] = 0.0
    w[5, 0, 1::7] = -0.0
    w[5, 1, 100:130] = float("nan")
    w[5, 1, 200:205] = float("inf")
    ref = R.Ref.of(cache, table)
    new_lens, kept, w_out = fa.cache_evict(cache, table, ln, w.cuda(), dst.cuda(), budget, recent)
    wl, wk, ww = ref.evict(np.array(lens), w.numpy(), dst.numpy(), budget, recent)
    assert np.array_equal(new_lens.cpu().numpy(), wl)
    assert np.array_equal(kept.cpu().numpy(), wk)
    assert np.array_equal(f64(w_out), ww, equal_nan=True)
    same_contents(cache, ref)
    fa.sync_status()


# ------------------------------------------------------------------ what the device refuses
def test_bad_pages_and_lengths_are_flagged():
    """Indexes that the host cannot see: nothing is followed out of bounds, the
    other sequences are right, and the next status says so."""
    fa = require_gpu()
    d, page, H, G = 64, 16, 2, 2
    lens = [40, 70, 33]
    cache, table, ln = R.make(fa, lens, H, d, page, seed=22)
    q = queries(3, H * G, 1, d, 23)
    ref = R.Ref.of(cache, table)
    want = ref.fwd(f64(q), lens, [1] * 3)
    fa.sync_status()

    def flagged():
        with pytest.raises(fa.Fa4Fp4Error) as e:
            fa.sync_status()
        assert e.value.status == 7
        fa.sync_status()

    good = np.zeros((3, H * G, 1), bool)
    good[[0, 2]] = True
    for bad_page in (-1, cache.num_pages, 1 << 30, -(1 << 31)):
        t = table.clone()
        t[1, 2] = bad_page
        o, lse = fa.cache_fwd(q, cache, t, ln, out_dtype=fa.OUT_F32)
        flagged()
        check_fwd(o, lse, want, d, True, good)
        # the page's keys count as absent
        sel = torch.tensor([0, 1, 3, 4], dtype=torch.int32, device="cuda").expand(3, H, 1, 4).contiguous()
        o1, _ = fa.cache_fwd(q, cache, table, ln, pages=sel, out_dtype=fa.OUT_F32)
        assert np.allclose(f64(o)[1], f64(o1)[1], rtol=1e-4, atol=1e-5)
        fa.cache_select(q, cache, t, ln, 2)
        flagged()
        fa.cache_weigh(q, lse, cache, t, ln, torch.zeros(3, H, table.shape[1] * page, device="cuda"))
        flagged()
        before = [x.clone() for x in (cache.k, cache.v)]
        fa.cache_append(cache, q[:, :H].contiguous(), q[:, :H].contiguous(), t, torch.tensor([1, 32, 0]).int().cuda(),
                        n_new=torch.tensor([0, 1, 0]).int().cuda())
        flagged()
        assert torch.equal(cache.k, before[0]) and torch.equal(cache.v, before[1])
        fa.cache_evict(cache, t, ln, torch.rand(3, H, table.shape[1] * page, device="cuda"),
                       torch.full((3, 2), bad_page, dtype=torch.int32, device="cuda"), 20, 0)
        flagged()
        assert torch.equal(cache.k, before[0]) and torch.equal(cache.v, before[1])
        fa.cache_fwd(q, cache, table, ln, pages=torch.full((3, H, 1, 2), max(bad_page, -5), dtype=torch.int32,
                                                           device="cuda") - (bad_page == -1) * 3)
        flagged()
    cap = table.shape[1] * page
    for bad_len in (-1, cap + 1, 1 << 30):
        x = ln.clone()
        x[1] = bad_len
        o, lse = fa.cache_fwd(q, cache, table, x, out_dtype=fa.OUT_F32)
        flagged()
        check_fwd(o, lse, want, d, True, good)
        fa.cache_weigh(q, lse, cache, table, x, torch.zeros(3, H, cap, device="cuda"))
        flagged()
        fa.cache_select(q, cache, table, x, 2)
        flagged()
    # no room left in the table: the tokens are not stored
    full = torch.tensor([0, cap - 1, 0]).int().cuda()
    kv = queries(3, H, 3, d, 24)
    fa.cache_append(cache, kv, kv, table, full, n_new=torch.tensor([0, 3, 0]).int().cuda())
    flagged()
    fa.cache_append(cache, kv, kv, table, full, n_new=torch.tensor([0, 4, 0]).int().cuda())
    flagged()


def test_refuses_wrong_tensors():
    fa = require_gpu()
    cache, table, ln = R.make(fa, [40, 70], 2, 64, 16)
    q = queries(2, 4, 1, 64, 25)
    bad = [dict(q=q[:, :, :, :32]), dict(q=q.float()), dict(q=q.cpu()), dict(q=queries(2, 4, 2, 64, 1)[:, :, :1]),
           dict(page_table=table.long()), dict(page_table=table.t()), dict(lens=ln[:1]), dict(lens=ln.cpu()),
           dict(out=torch.empty(2, 4, 1, 64, device="cuda")), dict(out_dtype=5),
           dict(pages=torch.zeros(2, 2, 1, 3, device="cuda")), dict(pages=torch.zeros(2, 1, 1, 3, device="cuda").int()),
           dict(workspace=torch.empty(1 << 20, device="cuda")), dict(q_lens=ln.float())]
    for kw in bad:
        args = dict(q=q, cache=cache, page_table=table, lens=ln)
        args.update(kw)
        with pytest.raises(ValueError):
            fa.cache_fwd(**args)
    with pytest.raises(fa.Fa4Fp4Error) as e:
        fa.cache_fwd(q, cache, table, ln, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 6
    with pytest.raises(fa.Fa4Fp4Error) as e:
        fa.cache_fwd(queries(2, 3, 1, 64, 1), cache, table, ln)
    assert e.value.status == 2
    with pytest.raises(fa.Fa4Fp4Error):
        fa.cache_evict(cache, table, ln, torch.zeros(2, 2, table.shape[1] * 16, device="cuda"), table, 0)
    with pytest.raises(ValueError):
        fa.cache_select(q, cache, table, ln, 0)
    fa.sync_status()


def test_empty_calls():
    fa = require_gpu()
    cache, table, ln = R.make(fa, [40], 2, 64, 16)
    t0, l0 = table[:0], ln[:0]
    e = queries(0, 4, 1, 64, 1)
    o, lse = fa.cache_fwd(e, cache, t0, l0)
    assert o.shape == (0, 4, 1, 64)
    fa.cache_append(cache, e[:, :2].contiguous(), e[:, :2].contiguous(), t0, l0)
    assert fa.cache_select(e, cache, t0, l0, 3).shape == (0, 2, 1, 3)
    z = queries(1, 4, 0, 64, 1)
    o, lse = fa.cache_fwd(z, cache, table, ln)
    assert o.shape == (1, 4, 0, 64) and lse.shape == (1, 4, 0)
    fa.sync_status()


# ------------------------------------------------------------------ together
def generate(fa, stream=None, graph=False):
    """A prompt, twelve decoding steps (the last eight sparse), eviction, four
    more steps; the queries and tokens are drawn.  Returns everything that came
    out, with the reference's values."""
    d, page, H, G, B = 64, 16, 2, 4, 3
    g = torch.Generator().manual_seed(30)
    prompt = torch.tensor([70, 1, 33], dtype=torch.int32)
    cache, table, _ = R.make(fa, [0] * B, H, d, page, seed=31, room=160, spare=20)
    used = set(table.flatten().tolist())
    free = torch.tensor([p for p in range(cache.num_pages) if p not in used], dtype=torch.int32)
    dst = free[:B * 5].view(B, 5).contiguous().cuda()
    kv = torch.randn(2, B, H, 70, d, generator=g).to(torch.bfloat16).cuda()
    qs = torch.randn(16, B, H * G, 1, d, generator=g).to(torch.bfloat16).cuda()
    ks, vs = (torch.randn(16, B, H, 1, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    out = []
    with torch.cuda.stream(stream or torch.cuda.current_stream()):
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        n = prompt.cuda()
        fa.cache_append(cache, kv[0].contiguous(), kv[1].contiguous(), table, lens, n_new=n)
        lens += n
        w = torch.zeros(B, H, table.shape[1] * page, device="cuda")
        q, k, v = qs[0].clone(), ks[0].clone(), vs[0].clone()

        def step(tb, weight, n_pages):
            fa.cache_append(cache, k, v, tb, lens)
            lens.add_(1)
            sel = fa.cache_select(q, cache, tb, lens, n_pages) if n_pages else None
            o, lse = fa.cache_fwd(q, cache, tb, lens, pages=sel, out_dtype=fa.OUT_F32)
            if weight is not None:
                # the weights are those of dense attention
                z = fa.cache_fwd(q, cache, tb, lens, out_dtype=fa.OUT_F32)[1] if n_pages else lse
                fa.cache_weigh(q, z, cache, tb, lens, weight)
            return o, lse

        def run(i, tb, weight, n_pages, g=None):
            q.copy_(qs[i]); k.copy_(ks[i]); v.copy_(vs[i])
            if g is not None:
                g[0].replay()
                return g[1]
            return step(tb, weight, n_pages)

        def capture(tb, weight, n_pages):
            if not graph:
                return None
            torch.cuda.current_stream().synchronize()
            cg = torch.cuda.CUDAGraph()
            with torch.cuda.graph(cg, stream=torch.cuda.current_stream() if stream else None):
                res = step(tb, weight, n_pages)
            return cg, res

        for lo, hi, tb, wt, n_pages in ((0, 4, table, w, 0), (4, 12, table, w, 3)):
            gr = capture(tb, wt, n_pages)
            for i in range(lo, hi):
                o, lse = run(i, tb, wt, n_pages, gr)
                out.append((o.clone(), lse.clone()))
        new_lens, kept, w2 = fa.cache_evict(cache, table, lens, w, dst, 40, 8)
        out.append((new_lens.clone(), kept.clone(), w2.clone()))
        lens.copy_(new_lens)
        gr = capture(dst, w2, 0)
        for i in range(12, 16):
            o, lse = run(i, dst, w2, 0, gr)
            out.append((o.clone(), lse.clone()))
        out.append((w.clone(), w2.clone(), lens.clone()))
    torch.cuda.synchronize()
    fa.sync_status()
    return out, cache, table, dst, (prompt, kv, qs, ks, vs)


def test_generation_against_reference():
    fa = require_gpu()
    out, cache, table, dst, (prompt, kv, qs, ks, vs) = generate(fa)
    H, d = cache.Hkv, cache.d
    empty, tb, _ = R.make(fa, [0] * 3, H, d, 16, seed=31, room=160, spare=20)
    assert torch.equal(tb, table)
    ref = R.Ref.of(empty, tb)
    lens = np.zeros(3, dtype=np.int64)
    ref.append(f64(kv[0]), f64(kv[1]), lens, prompt.numpy())
    lens += prompt.numpy()
    one = [1, 1, 1]
    for i in range(12):
        ref.append(f64(ks[i]), f64(vs[i]), lens, one)
        lens += 1
        q = f64(qs[i])
        pages = ref.select(q, lens, one, 3) if i >= 4 else None
        check_fwd(*out[i], ref.fwd(q, lens, one, pages=pages), d, True)
    new_lens, kept, w2 = out[12]
    w = f64(out[-1][0])
    # the kept tokens follow from the weights that the GPU accumulated
    wl, wk, ww = ref.evict(lens, w, dst.cpu().numpy(), 40, 8)
    assert np.array_equal(new_lens.cpu().numpy(), wl) and np.array_equal(kept.cpu().numpy(), wk)
    assert np.array_equal(f64(w2), ww)
    ref.table, lens = dst.cpu().numpy(), wl
    for i in range(12, 16):
        ref.append(f64(ks[i]), f64(vs[i]), lens, one)
        lens = lens + 1
        check_fwd(*out[13 + i - 12], ref.fwd(f64(qs[i]), lens, one), d, True)
    same_contents(cache, ref)
    # every query spreads a weight of one over what it sees: 12 steps, 4 heads a kv head
    assert np.allclose(w.sum(-1), 12 * 4, rtol=1e-5)


@pytest.mark.parametrize("side,graph", [(True, False), (True, True)])
def test_generation_on_a_stream_and_from_graphs(side, graph):
    """Bit for bit what the default stream gives, from another stream and from
    captured and replayed steps."""
    fa = require_gpu()
    want = generate(fa)[0]
    got = generate(fa, torch.cuda.Stream() if side else None, graph)[0]
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_two_streams_at_once():
    """Two calls in flight, each with its own workspace."""
    fa = require_gpu()
    cache, table, ln = R.make(fa, [9000, 40], 2, 128, 64, seed=33)
    q = queries(2, 8, 1, 128, 34)
    want = fa.cache_fwd(q, cache, table, ln)
    sel = fa.cache_select(q, cache, table, ln, 9)
    want_s = fa.cache_fwd(q, cache, table, ln, pages=sel)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        with torch.cuda.stream(s1):
            got.append((want, fa.cache_fwd(q, cache, table, ln)))
        with torch.cuda.stream(s2):
            got.append((want_s, fa.cache_fwd(q, cache, table, ln, pages=fa.cache_select(q, cache, table, ln, 9))))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    fa.sync_status()
