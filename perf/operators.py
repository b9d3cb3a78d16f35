"""The 8-bit key/value cache operators, as timed cases.

Every case is one pass through one operator on a paged cache whose pages hold
E4M3 codes with one power-of-two scale per page and head: ``append`` (new
tokens into the cache), ``fwd`` (attention over the cache), ``sparse`` (page
selection and attention over the selected pages), ``weigh`` (attention weight
that each cached token received) and ``evict`` (the heaviest and the newest
tokens copied into fresh pages).

``own = False`` runs each operator in elementary torch operations, ``own =
True`` through this package; both take the same state.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    c = []
    # one decoding step of a serving batch: a token for each of 64 sequences
    c.append(dict(name="append_token", op="append", B=64, Hkv=8, d=128, page=64, T=1, lo=1, hi=2047, ragged=False))
    # two prompts of the training length go into an empty cache
    c.append(dict(name="append_prompt", op="append", B=2, Hkv=8, d=128, page=64, T=8192, lo=0, hi=0, ragged=False))
    # one user, a short conversation: latency
    c.append(dict(name="fwd_one", op="fwd", B=1, Hq=32, Hkv=8, d=128, page=64, T=1, lo=1000, hi=1000, ragged=False,
                  f32=False))
    # a serving batch of mixed lengths, one token each: bandwidth
    c.append(dict(name="fwd_batch", op="fwd", B=64, Hq=32, Hkv=8, d=128, page=64, T=1, lo=1, hi=8192, ragged=False,
                  f32=False))
    # drafted tokens (up to four a sequence) checked against long contexts, FP32 output, heads of 64
    c.append(dict(name="fwd_draft", op="fwd", B=4, Hq=24, Hkv=8, d=64, page=32, T=4, lo=16001, hi=32760, ragged=True,
                  f32=True))
    # a chunk of a prompt of 8192 tokens over what was cached before
    c.append(dict(name="fwd_chunk", op="fwd", B=2, Hq=32, Hkv=8, d=128, page=64, T=1024, lo=8192, hi=8192,
                  ragged=False, f32=False))
    # long contexts read sparsely: 64 pages of 512
    c.append(dict(name="sparse_long", op="sparse", B=8, Hq=32, Hkv=8, d=128, page=64, T=1, lo=24001, hi=32768,
                  ragged=False, pages=64))
    # small pages, one kv head per query head, a few drafted tokens
    c.append(dict(name="sparse_draft", op="sparse", B=2, Hq=16, Hkv=16, d=64, page=16, T=3, lo=5001, hi=8192,
                  ragged=True, pages=40))
    # statistics of one decoding step of a batch
    c.append(dict(name="weigh_token", op="weigh", B=16, Hq=32, Hkv=8, d=128, page=64, T=1, lo=4001, hi=8192,
                  ragged=False))
    # statistics of the last part of a prompt
    c.append(dict(name="weigh_chunk", op="weigh", B=2, Hq=32, Hkv=8, d=128, page=64, T=256, lo=4096, hi=4096,
                  ragged=False))
    # one conversation cut back to a thousand tokens
    c.append(dict(name="evict_one", op="evict", B=1, Hkv=8, d=128, page=64, lo=4096, hi=4096, budget=1000, recent=64))
    # a batch cut back to half
    c.append(dict(name="evict_batch", op="evict", B=16, Hkv=8, d=128, page=64, lo=4001, hi=8192, budget=4096,
                  recent=256))
    return c


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "fwd", "fwd", "sparse", "weigh", "evict"])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    if op == "append":
        T = _log(rng, 1, 8192)
        B = _log(rng, 1, max(1, min(64, 16384 // T)))
        hi = 0 if rng.random() < 0.2 else _log(rng, 1, 2047)
        return dict(op=op, B=B, Hkv=min(Hkv, 8), d=d, page=page, T=T, lo=0, hi=hi, ragged=rng.random() < 0.5)
    if op == "evict":
        B = _log(rng, 1, 16)
        hi = _log(rng, 100, 8192)
        budget = _log(rng, 16, max(16, hi))
        return dict(op=op, B=B, Hkv=min(Hkv, 8), d=d, page=page, lo=rng.randint(1, hi), hi=hi, budget=budget,
                    recent=rng.randint(0, budget))
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    Hq = min(Hkv * G, 32) // Hkv * Hkv
    if op == "sparse":
        T = rng.choice([1, 1, 1, 2, 3, 5])
        hi = _log(rng, 500, 32768)
        B = _log(rng, 1, max(1, 8 * 32768 // (hi * T)) if hi * T > 32768 else 8)
        return dict(op=op, B=B, Hq=Hq, Hkv=min(Hkv, 8) if Hq % 8 == 0 else Hkv, d=d, page=page, T=T,
                    lo=rng.randint(T, hi), hi=hi, ragged=T > 1, pages=_log(rng, 2, max(2, 4096 // page)))
    if op == "weigh":
        T = _log(rng, 1, 256)
        hi = _log(rng, max(T, 64), 4096 if T > 8 else 8192)
        B = _log(rng, 1, 2 if T > 8 else 16)
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, T=T, lo=rng.randint(T, hi), hi=hi, ragged=T > 1)
    T = 1 if rng.random() < 0.5 else _log(rng, 2, 1024)
    hi = _log(rng, max(T, 64), 8192 if T > 8 else 32768)
    B = _log(rng, 1, max(1, min(64, 2 * 1024 * 8192 // (T * hi)))) if T > 8 else _log(rng, 1, max(1, min(64, 524288 // hi // 4)))
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, T=T, lo=rng.randint(T, hi), hi=hi, ragged=T > 1,
                f32=T <= 8 and rng.random() < 0.4)


# ----------------------------------------------------------------------------
# state
# ----------------------------------------------------------------------------
def _exponent(amax):
    """The least X with amax <= 448 * 2^X, at least -127 (amax FP32)."""
    m, e = torch.frexp(amax)
    return torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-127).where(amax > 0, torch.full_like(e, -127))


def _pow2(x):
    """2^x in FP32 for integer x up to 127, subnormals included (0 below -149), by its bits."""
    x = x.int()
    low = torch.ones_like(x) << (x + 149).clamp(0, 22)
    return torch.where(x >= -126, (x.clamp(min=-126) + 127) << 23, low.masked_fill(x < -149, 0)).view(torch.float32)


def _codes(x, X):
    """E4M3 codes of x * 2^-X (X broadcast against x)."""
    return (x * _pow2(-X)).to(torch.float8_e4m3fn)


def _values(codes, X):
    """FP32 values of E4M3 codes under the exponents X."""
    return codes.view(torch.float8_e4m3fn).float() * _pow2(X)


def _kv(g, shape, outliers):
    x = torch.randn(shape, generator=g, device=DEV)
    if outliers:      # a few channels carry most of a key's magnitude
        x[..., : max(1, shape[-1] // 32)] *= 8.0
    return x.to(torch.bfloat16)


def _lens(g, case):
    return torch.randint(case["lo"], case["hi"] + 1, (case["B"],), generator=g, device=DEV).int()


def _pool(case, g, room):
    """An empty cache for B sequences of up to `room` tokens, its pages in random order."""
    B, H, d, P = case["B"], case["Hkv"], case["d"], case["page"]
    per = max(1, -(-room // P))
    n = B * per
    u8 = dict(dtype=torch.uint8, device=DEV)
    st = dict(kc=torch.zeros((n, H, P, d), **u8), vc=torch.zeros((n, H, P, d), **u8), ks=torch.zeros((n, H), **u8),
              vs=torch.zeros((n, H), **u8), kb=torch.zeros((n, H, 2, d), **u8))
    st["table"] = torch.randperm(n, generator=g, device=DEV).int().view(B, per)
    return st


def _fill(st, case, g, lens):
    """Random tokens into the cache, a sequence at a time."""
    B, H, d, P = case["B"], case["Hkv"], case["d"], case["page"]
    per = st["table"].shape[1]
    pos = torch.arange(per * P, device=DEV).view(per, 1, P, 1)
    for b in range(B):
        at = st["table"][b].long()
        there = pos < lens[b]
        for name, outliers in (("k", True), ("v", False)):
            x = _kv(g, (per, H, P, d), outliers).float().where(there, torch.zeros((), device=DEV))
            X = _exponent(x.abs().amax((2, 3)))
            c = _codes(x, X[:, :, None, None])
            st[name + "c"][at] = c.view(torch.uint8)
            st[name + "s"][at] = (X + 127).to(torch.uint8)
            if name == "k":
                f = c.float()
                lo = f.where(there, torch.full_like(f, 448.0)).amin(2)
                hi = f.where(there, torch.full_like(f, -448.0)).amax(2)
                st["kb"][at] = torch.stack([lo, hi], 2).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, H, d, P = case["B"], case["Hkv"], case["d"], case["page"]
    lens = _lens(g, case)
    if case["op"] == "append":
        T = case["T"]
        st = _pool(case, g, case["hi"] + T)
        _fill(st, case, g, lens)
        st["k"] = _kv(g, (B, H, T, d), True)
        st["v"] = _kv(g, (B, H, T, d), False)
        st["n_new"] = torch.randint(0, T + 1, (B,), generator=g, device=DEV).int() if case["ragged"] else None
        st.update(case=case, lens=lens)
        return st
    st = _pool(case, g, case["hi"])
    _fill(st, case, g, lens)
    st.update(case=case, lens=lens)
    per = st["table"].shape[1]
    if case["op"] == "evict":
        room = -(-case["budget"] // P)
        n = st["kc"].shape[0]
        # the fresh pages lie in the same pool, behind the others
        for k in ("kc", "vc", "ks", "vs", "kb"):
            st[k] = torch.cat([st[k], torch.zeros((B * room, *st[k].shape[1:]), dtype=torch.uint8, device=DEV)])
        st["dst"] = (n + torch.randperm(B * room, generator=g, device=DEV)).int().view(B, room)
        # accumulated weights fall off like 1/rank in random order
        st["w"] = 1.0 / (torch.rand((B, H, per * P), generator=g, device=DEV) + 1e-4)
        return st
    T = case["T"]
    st["q"] = torch.randn((B, case["Hq"], T, d), generator=g, device=DEV).to(torch.bfloat16)
    st["q_lens"] = torch.randint(1, T + 1, (B,), generator=g, device=DEV).int() if case["ragged"] else None
    if case["op"] == "weigh":
        st["lse"] = _attend(st)[1].where(_rows(st), torch.zeros((), device=DEV)).contiguous()
        st["w"] = torch.rand((B, H, per * P), generator=g, device=DEV)
        st["w_out"] = torch.zeros((B, H, per * P), device=DEV)
        return st
    st["o"] = torch.zeros((B, case["Hq"], T, d), device=DEV,
                          dtype=torch.float32 if case.get("f32") else torch.bfloat16)
    st["lse"] = torch.zeros((B, case["Hq"], T), device=DEV)
    return st


# ----------------------------------------------------------------------------
# the operators in elementary operations
# ----------------------------------------------------------------------------
def _visible(st):
    """[B, T]: how many keys token t of each sequence sees (at least 0)."""
    T = st["q"].shape[2]
    n = st["q_lens"] if st["q_lens"] is not None else torch.full_like(st["lens"], T)
    t = torch.arange(T, device=DEV)
    return (st["lens"][:, None] - n[:, None] + t + 1).clamp(min=0).minimum(st["lens"][:, None])


def _rows(st):
    """[B, 1, T]: the rows that hold a token."""
    T = st["q"].shape[2]
    t = torch.arange(T, device=DEV)
    n = st["q_lens"] if st["q_lens"] is not None else torch.full_like(st["lens"], T)
    return (t < n[:, None])[:, None, :]


def _pages(st, at):
    """K and V of the physical pages `at` [..., n]: FP32 [..., H, n * P, d]."""
    out = []
    for name in ("k", "v"):
        x = _values(st[name + "c"][at], (st[name + "s"][at].int() - 127)[..., None, None])   # [..., n, H, P, d]
        x = x.movedim(-3, -4)
        out.append(x.flatten(-3, -2))
    return out


def _softmax_v(s, V):
    """s [..., R, L] with -inf where masked, V [..., L, d]: (o, lse); rows without a key give 0 and -inf."""
    m = s.amax(-1, keepdim=True)
    m = m.where(m > -math.inf, torch.zeros((), device=DEV))
    e = torch.exp(s - m)
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e, V) / l.where(l > 0, torch.ones((), device=DEV))
    return o, (m + torch.log(l)).squeeze(-1)


def _scores(st):
    """(s [B, H, G * T, L] masked with -inf, V [B, H, L, d]) over all pages of the table."""
    case, q = st["case"], st["q"]
    B, Hq, T, d = q.shape
    H = case["Hkv"]
    K, V = _pages(st, st["table"].long())
    L = K.shape[-2]
    pos = torch.arange(L, device=DEV)
    V = V.where((pos < st["lens"][:, None])[:, None, :, None], torch.zeros((), device=DEV))
    s = torch.matmul(q.float().view(B, H, Hq // H * T, d), K.transpose(-1, -2)) / math.sqrt(d)
    see = (pos < _visible(st)[..., None])[:, None, None]                   # [B, 1, 1, T, L]
    s = s.view(B, H, Hq // H, T, L).masked_fill(~see, -math.inf)
    return s.view(B, H, Hq // H * T, L), V


def _attend(st):
    B, Hq, T, d = st["q"].shape
    s, V = _scores(st)
    o, lse = _softmax_v(s, V)
    return o.view(B, Hq, T, d), lse.view(B, Hq, T)


def _fwd(st):
    o, lse = _attend(st)
    rows = _rows(st)
    return o.to(st["o"].dtype).where(rows[..., None], st["o"]), lse.where(rows, st["lse"])


def _select(st):
    """The pages with the highest upper bound of q.k, summed over the query heads of a kv head, in 64 bits."""
    case, q = st["case"], st["q"]
    B, Hq, T, d = q.shape
    H, P, n = case["Hkv"], case["page"], case["pages"]
    at = st["table"].long()
    X = st["ks"][at].int() - 127                                           # [B, per, H]
    kb = st["kb"][at].view(torch.float8_e4m3fn).double() * torch.exp2(X.double())[..., None, None]
    qg = q.double().view(B, H, Hq // H, T, d)
    up, dn = qg.clamp(min=0).sum(2), qg.clamp(max=0).sum(2)                # [B, H, T, d]
    kb = kb.permute(0, 2, 3, 4, 1)                                         # [B, H, 2, d, per]
    score = torch.matmul(up, kb[:, :, 1]) + torch.matmul(dn, kb[:, :, 0])  # [B, H, T, per]
    per = score.shape[-1]
    count = (_visible(st) + P - 1) // P                                    # [B, T]
    page = torch.arange(per, device=DEV)
    score = score.masked_fill(page >= count[:, None, :, None], -math.inf)
    score = score.masked_fill(page == count[:, None, :, None] - 1, math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., : n]
    if order.shape[-1] < n:
        order = torch.cat([order, order.new_full((*order.shape[:-1], n - order.shape[-1]), per)], -1)
    rank = torch.arange(n, device=DEV)
    order = order.masked_fill(rank >= count[:, None, :, None], per)
    order = torch.sort(order, dim=-1)[0]
    return order.masked_fill(order >= per, -1).int().masked_fill(~_rows(st)[..., None], -1)


def _sparse(st):
    case, q = st["case"], st["q"]
    B, Hq, T, d = q.shape
    H, P, n = case["Hkv"], case["page"], case["pages"]
    sel = _select(st)                                                      # [B, H, T, n]
    there = sel >= 0
    lp = sel.clamp(min=0).long()
    at = st["table"].long()[:, None, None].expand(B, H, T, -1).gather(-1, lp)
    h = torch.arange(H, device=DEV)[None, :, None, None]
    kv = []
    for name in ("k", "v"):
        X = (st[name + "s"][at, h].int() - 127)[..., None, None]
        kv.append(_values(st[name + "c"][at, h], X).flatten(-3, -2))       # [B, H, T, n * P, d]
    K, V = kv
    pos = (lp[..., None] * P + torch.arange(P, device=DEV)).flatten(-2)    # [B, H, T, n * P]
    there = there[..., None].expand(*there.shape, P).flatten(-2)
    see = there & (pos < _visible(st)[:, None, :, None])
    V = V.where(see[..., None], torch.zeros((), device=DEV))
    qg = q.float().view(B, H, Hq // H, T, d).transpose(2, 3)               # [B, H, T, G, d]
    s = torch.matmul(qg, K.transpose(-1, -2)) / math.sqrt(d)
    o, lse = _softmax_v(s.masked_fill(~see[..., None, :], -math.inf), V)
    o = o.transpose(2, 3).reshape(B, Hq, T, d)
    lse = lse.transpose(2, 3).reshape(B, Hq, T)
    rows = _rows(st)
    return sel, o.to(st["o"].dtype).where(rows[..., None], st["o"]), lse.where(rows, st["lse"])


def _weigh(st):
    case, q = st["case"], st["q"]
    B, Hq, T, d = q.shape
    H = case["Hkv"]
    s, _ = _scores(st)
    L = s.shape[-1]
    lse = st["lse"].view(B, H, Hq // H * T, 1)
    use = (lse > -math.inf) & _rows(st).expand(B, Hq, T).reshape(B, H, Hq // H * T, 1)
    p = torch.exp(s - lse.where(use, torch.zeros((), device=DEV))).where(use, torch.zeros((), device=DEV))
    w = st["w"] + p.sum(2)
    return w.where((torch.arange(L, device=DEV) < st["lens"][:, None])[:, None], st["w_out"])


def _append(st):
    case = st["case"]
    B, H, d, P, T = (case[k] for k in ("B", "Hkv", "d", "page", "T"))
    lens = st["lens"]
    n = st["n_new"] if st["n_new"] is not None else torch.full_like(lens, T)
    per = st["table"].shape[1]
    first = lens // P
    last = ((lens + n - 1).maximum(lens) // P).clamp(max=per - 1)
    j = torch.arange((T + P - 1) // P + 1, device=DEV)
    lp = (first[:, None] + j).minimum(last[:, None])                       # [B, J] logical pages
    at = st["table"].long().gather(1, lp.long())                           # [B, J] physical pages
    pos = lp[..., None] * P + torch.arange(P, device=DEV)                  # [B, J, P]
    end = (lens + n)[:, None, None]
    new = (pos >= lens[:, None, None]) & (pos < end)
    old = pos < lens[:, None, None]
    touched = new.any(-1)                                                  # [B, J]
    src = (pos - lens[:, None, None]).clamp(0, T - 1).long()
    bi = torch.arange(B, device=DEV)[:, None, None]
    for name in ("k", "v"):
        x = st[name].float().transpose(1, 2)[bi, src]                      # [B, J, P, H, d]
        x = x.permute(0, 1, 3, 2, 4)                                       # [B, J, H, P, d]
        isnew, isold = new[:, :, None, :, None], old[:, :, None, :, None]
        had = st[name + "c"][at]                                           # [B, J, H, P, d]
        Xo = st[name + "s"][at].int() - 127                                # [B, J, H]
        X = _exponent(x.abs().where(isnew, torch.zeros((), device=DEV)).amax((-1, -2)))
        X = X.maximum(Xo.where(old.any(-1)[..., None], torch.full_like(Xo, -127)))
        X = X.where(touched[..., None], Xo)
        c_new = _codes(x, X[..., None, None])
        c_old = (had.view(torch.float8_e4m3fn).float() * _pow2(Xo - X)[..., None, None]).to(torch.float8_e4m3fn)
        c = torch.where(isnew, c_new.view(torch.uint8), torch.where(isold, c_old.view(torch.uint8), had))
        st[name + "c"][at] = c
        st[name + "s"][at] = (X + 127).to(torch.uint8)
        if name == "k":
            f = c.view(torch.float8_e4m3fn).float()
            lo = f.where(isnew | isold, torch.full_like(f, 448.0)).amin(-2)
            hi = f.where(isnew | isold, torch.full_like(f, -448.0)).amax(-2)
            kb = torch.stack([lo, hi], -2).to(torch.float8_e4m3fn).view(torch.uint8)
            st["kb"][at] = kb.where(touched[..., None, None, None], st["kb"][at])


def _evict(st):
    case = st["case"]
    B, H, d, P, n, recent = (case[k] for k in ("B", "Hkv", "d", "page", "budget", "recent"))
    lens, w = st["lens"], st["w"]
    L = w.shape[-1]
    pos = torch.arange(L, device=DEV)
    there = (pos < lens[:, None])[:, None]
    newest = (pos >= (lens - recent)[:, None])[:, None]
    key = w.masked_fill(newest, math.inf).masked_fill(~there, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True)[1][..., : n]
    if order.shape[-1] < n:
        order = torch.cat([order, order.new_full((B, H, n - order.shape[-1]), L)], -1)
    new_lens = lens.clamp(max=n)
    order = order.masked_fill(torch.arange(n, device=DEV) >= new_lens[:, None, None], L)
    kept = torch.sort(order, dim=-1)[0]
    valid = kept < L
    src = kept.clamp(max=L - 1)
    room = st["dst"].shape[1]
    pad = room * P - n
    h = torch.arange(H, device=DEV)[None, :, None]
    at = st["table"].long()[:, None].expand(B, H, -1).gather(-1, src // P)
    dst = st["dst"].long()                                                 # [B, room]
    v4 = torch.cat([valid, valid.new_zeros((B, H, pad))], -1).view(B, H, room, P)
    for name in ("k", "v"):
        x = _values(st[name + "c"][at, h, src % P], (st[name + "s"][at, h].int() - 127)[..., None])
        x = torch.cat([x, x.new_zeros((B, H, pad, d))], 2).view(B, H, room, P, d)
        x = x.where(v4[..., None], torch.zeros((), device=DEV))
        X = _exponent(x.abs().amax((-1, -2)))
        c = _codes(x, X[..., None, None])
        had = st[name + "c"][dst].transpose(1, 2)
        st[name + "c"][dst] = torch.where(v4[..., None], c.view(torch.uint8), had).transpose(1, 2)
        used = v4.any(-1)
        st[name + "s"][dst] = torch.where(used, (X + 127).to(torch.uint8), st[name + "s"][dst].transpose(1, 2)).transpose(1, 2)
        if name == "k":
            f = c.float()
            lo = f.where(v4[..., None], torch.full_like(f, 448.0)).amin(-2)
            hi = f.where(v4[..., None], torch.full_like(f, -448.0)).amax(-2)
            kb = torch.stack([lo, hi], -2).to(torch.float8_e4m3fn).view(torch.uint8)    # [B, H, room, 2, d]
            kb = kb.where(used[..., None, None], st["kb"][dst].transpose(1, 2))
            st["kb"][dst] = kb.transpose(1, 2)
    w_out = torch.cat([w.gather(-1, src).where(valid, torch.zeros((), device=DEV)), w.new_zeros((B, H, pad))], -1)
    return new_lens, kept.masked_fill(~valid, -1).int(), w_out


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def _contents(st):
    """The cache as values: codes as E4M3 numbers, exponents as whole numbers."""
    f8 = torch.float8_e4m3fn
    return dict(k=st["kc"].view(f8), v=st["vc"].view(f8), ks=st["ks"], vs=st["vs"], kb=st["kb"].view(f8))


def _own(st):
    import precision_attention_fa4fp4_gb300 as fa
    op = st["case"]["op"]
    cache = fa.KVCache(st["kc"], st["vc"], st["ks"], st["vs"], st["kb"])
    if op == "append":
        fa.cache_append(cache, st["k"], st["v"], st["table"], st["lens"], n_new=st["n_new"])
        return _contents(st)
    if op == "fwd":
        return fa.cache_fwd(st["q"], cache, st["table"], st["lens"], q_lens=st["q_lens"], causal=True,
                            out_dtype=fa.OUT_F32 if st["case"]["f32"] else fa.OUT_BF16, out=st["o"], lse=st["lse"])
    if op == "sparse":
        sel = fa.cache_select(st["q"], cache, st["table"], st["lens"], st["case"]["pages"], q_lens=st["q_lens"])
        o, lse = fa.cache_fwd(st["q"], cache, st["table"], st["lens"], q_lens=st["q_lens"], causal=True,
                              out=st["o"], lse=st["lse"], pages=sel)
        return sel, o, lse
    if op == "weigh":
        return fa.cache_weigh(st["q"], st["lse"], cache, st["table"], st["lens"], st["w"], q_lens=st["q_lens"],
                              causal=True, out=st["w_out"])
    new_lens, kept, w_out = fa.cache_evict(cache, st["table"], st["lens"], st["w"], st["dst"], st["case"]["budget"],
                                           st["case"]["recent"])
    return dict(_contents(st), lens=new_lens, kept=kept, w=w_out)


def run(st):
    if own:
        return _own(st)
    op = st["case"]["op"]
    if op == "append":
        _append(st)
        return _contents(st)
    if op == "fwd":
        return _fwd(st)
    if op == "sparse":
        return _sparse(st)
    if op == "weigh":
        return _weigh(st)
    new_lens, kept, w_out = _evict(st)
    return dict(_contents(st), lens=new_lens, kept=kept, w=w_out)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    B, H, d, P = case["B"], case["Hkv"], case["d"], case["page"]
    L = (case["lo"] + case["hi"]) / 2                     # tokens of an average sequence
    head = 2 * d + 2.0 / P                                # bytes of one cached token of one head
    if case["op"] == "append":
        new = case["T"] / 2 if case["ragged"] else case["T"]
        return dict(bytes=B * H * new * (4 * d + head), flops=0)
    if case["op"] == "evict":
        kept = min(L, case["budget"])
        return dict(bytes=B * H * (4 * L + kept * (2 * head + 8)), flops=0)
    Hq, T = case["Hq"], case["T"]
    if case["ragged"]:
        T = (1 + T) / 2
    see = max(0.0, L - (T - 1) / 2)                       # keys that an average token sees
    rows = B * Hq * T
    if case["op"] == "fwd":
        return dict(bytes=B * H * L * head + rows * d * (6 if case["f32"] else 4) + 4 * rows, flops=4 * rows * see * d)
    if case["op"] == "weigh":
        return dict(bytes=B * H * L * (d + 1.0 / P + 8) + rows * (2 * d + 4), flops=2 * rows * see * d)
    pages = min(case["pages"], see / P)
    return dict(bytes=B * H * (L / P) * (2 * d + 1) + B * H * T * (pages * P * head + 4 * pages) + rows * (4 * d + 4),
                flops=4 * rows * pages * P * d + 4 * B * H * T * (see / P) * d)


# ----------------------------------------------------------------------------
# the operators in 64 bits, from their definitions, a sequence at a time
# ----------------------------------------------------------------------------
def _table64():
    """The 256 E4M3 values from their bit fields."""
    out = []
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out.append(float("nan") if (e == 15 and m == 7) else (-v if s else v))
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def _read64(st, name, table_row, length, tab):
    """Tokens 0..length-1 of one sequence: [H, length, d] in 64 bits."""
    P = st["case"]["page"]
    at = table_row[: -(-length // P)].long()
    x = tab[st[name + "c"][at].long()] * torch.exp2(st[name + "s"][at].double() - 127)[:, :, None, None]
    return x.transpose(0, 1).flatten(1, 2)[:, :length]


def _round64(x):
    """To the nearest E4M3 value, ties to even (|x| <= 448)."""
    e = torch.frexp(x)[1].double() - 1
    step = torch.exp2(e.clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exponent64(amax):
    """ceil(log2(amax / 448)), at least -127, by comparisons."""
    X = torch.full_like(amax, -127.0)
    guess = torch.floor(torch.log2(amax.clamp(min=1e-60) / 448)) - 1
    for k in range(4):
        X = torch.where((amax > 448 * torch.exp2(X)) & (guess + k > X), guess + k, X)
    return X


def exact(case, seed):
    st = prepare(case, seed)
    tab = _table64()
    B, H, d, P = case["B"], case["Hkv"], case["d"], case["page"]
    lens = st["lens"].tolist()
    if case["op"] in ("append", "evict"):
        out = dict(k=tab[st["kc"].long()], v=tab[st["vc"].long()], ks=st["ks"].long(), vs=st["vs"].long(),
                   kb=tab[st["kb"].long()])

        def store(name, page, h_values, floor):
            """h_values [H, n, d] become the first n tokens of `page`, under at least the exponents `floor` [H]."""
            X = torch.maximum(_exponent64(h_values.abs().amax((1, 2))), floor)
            c = _round64(h_values * torch.exp2(-X)[:, None, None])
            out[name][page, :, : c.shape[1]] = c
            out[name + "s"][page] = (X + 127).long()
            if name == "k":
                out["kb"][page, :, 0], out["kb"][page, :, 1] = c.amin(1), c.amax(1)

    if case["op"] == "append":
        low = torch.full((H,), -127.0, dtype=torch.float64, device=DEV)
        for b in range(B):
            n = case["T"] if st["n_new"] is None else int(st["n_new"][b])
            if n == 0:
                continue
            for name in ("k", "v"):
                start = lens[b] // P * P
                had = _read64(st, name, st["table"][b], lens[b], tab)[:, start:]
                x = torch.cat([had, st[name][b, :, :n].double()], 1)
                for i in range(0, x.shape[1], P):
                    page = int(st["table"][b, (start + i) // P])
                    part = i == 0 and had.shape[1] > 0
                    store(name, page, x[:, i: i + P], st[name + "s"][page].double() - 127 if part else low)
        return out
    if case["op"] == "evict":
        n, recent = case["budget"], case["recent"]
        kept = torch.full((B, H, n), -1, dtype=torch.int64, device=DEV)
        w_out = torch.zeros((B, H, st["dst"].shape[1] * P), dtype=torch.float64, device=DEV)
        low = torch.full((H,), -127.0, dtype=torch.float64, device=DEV)
        for b in range(B):
            L = lens[b]
            m = min(L, n)
            w = st["w"][b, :, :L].double().clone()
            w[:, max(0, L - recent):] = math.inf
            at = torch.sort(torch.argsort(-w, dim=-1, stable=True)[:, :m], dim=-1)[0]
            kept[b, :, :m] = at
            w_out[b, :, :m] = st["w"][b, :, :L].double().gather(1, at)
            for name in ("k", "v"):
                x = _read64(st, name, st["table"][b], L, tab).gather(1, at[..., None].expand(-1, -1, d))
                for i in range(0, m, P):
                    store(name, int(st["dst"][b, i // P]), x[:, i: i + P], low)
        return dict(out, lens=torch.tensor([min(x, n) for x in lens]), kept=kept, w=w_out)
    q, Hq, T = st["q"].double(), case["Hq"], case["T"]
    G = Hq // H
    o = torch.zeros((B, Hq, T, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, Hq, T), dtype=torch.float64, device=DEV)
    sel = torch.full((B, H, T, case.get("pages", 0)), -1, dtype=torch.int64, device=DEV)
    w = st["w_out"].double() if case["op"] == "weigh" else None
    for b in range(B):
        L = lens[b]
        n = T if st["q_lens"] is None else int(st["q_lens"][b])
        K = _read64(st, "k", st["table"][b], L, tab)
        V = _read64(st, "v", st["table"][b], L, tab) if case["op"] != "weigh" else None
        if case["op"] == "weigh":
            w[b, :, :L] = st["w"][b, :, :L].double()
        if case["op"] == "sparse":
            at = st["table"][b, : -(-L // P)].long()
            kb = tab[st["kb"][at].long()] * torch.exp2(st["ks"][at].double() - 127)[:, :, None, None]
        for h in range(H):
            x = q[b, h * G: (h + 1) * G, :n]                               # [G, n, d]
            see = L - n + 1 + torch.arange(n, device=DEV)
            s = torch.matmul(x, K[h].T) / math.sqrt(d)                     # [G, n, L]
            hide = torch.arange(L, device=DEV) >= see[:, None]
            if case["op"] == "sparse":
                for t in range(n):
                    c = -(-max(0, int(see[t])) // P)
                    if c == 0:
                        continue
                    bound = torch.maximum(x[:, t, None] * kb[:c, h, 0], x[:, t, None] * kb[:c, h, 1]).sum((0, 2))
                    bound[c - 1] = math.inf
                    top = torch.sort(torch.argsort(-bound, stable=True)[: case["pages"]])[0]
                    sel[b, h, t, : len(top)] = top
                    keep = torch.zeros(-(-L // P), dtype=torch.bool, device=DEV)
                    keep[top] = True
                    hide[t] |= ~keep.repeat_interleave(P)[:L]
            s = s.masked_fill(hide, -math.inf)
            if case["op"] == "weigh":
                z = st["lse"][b, h * G: (h + 1) * G, :n].double()
                w[b, h, :L] += torch.exp(s - z[..., None]).where(z[..., None] > -math.inf, torch.zeros((), device=DEV, dtype=torch.float64)).sum((0, 1))
                continue
            z = torch.logsumexp(s, -1)
            lse[b, h * G: (h + 1) * G, :n] = z
            p = torch.exp(s - z[..., None]).where(z[..., None] > -math.inf, torch.zeros((), device=DEV, dtype=torch.float64))
            o[b, h * G: (h + 1) * G, :n] = torch.matmul(p, V[h])
    if case["op"] == "weigh":
        return w
    return (o, lse) if case["op"] == "fwd" else (sel, o, lse)


if __name__ == "__main__":
    r = random.Random(0)
    for c in listed() + [draw(r) for _ in range(6)]:
        print(c, work(c))
