"""The 8-bit cache operators in plain 64-bit numpy, one sequence, head and token
at a time: the reference of the cache tests.  Shares nothing with the package."""
import numpy as np
import torch


def _values():
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if (c & 0x7f) == 0x7f else (-v if s else v)
    return out


E4M3 = _values()
_POS = E4M3[:127]                      # 0 .. 448, ascending


def e4m3_codes(x):
    """Nearest E4M3 code, ties to the even code, saturating; the sign of zero kept."""
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (c + 128 * np.signbit(x)).astype(np.uint8)


def least_exponent(amax):
    """The least integer X >= -127 with amax <= 448 * 2^X."""
    X = -127
    while amax > 448 * 2.0 ** X:
        X += 1
    return X


class Ref:
    """The pool and the page tables on the host."""

    def __init__(self, k, v, ks, vs, kb, table):
        self.k, self.v, self.ks, self.vs, self.kb, self.table = (np.array(x) for x in (k, v, ks, vs, kb, table))
        self.page, self.d, self.H = self.k.shape[2], self.k.shape[3], self.k.shape[1]

    @classmethod
    def of(cls, cache, table):
        return cls(*(t.cpu().numpy() for t in (cache.k, cache.v, cache.ks, cache.vs, cache.kb)), table.cpu().numpy())

    def read(self, name, b, h, n):
        """Values of tokens 0..n-1: [n, d]."""
        P = self.page
        codes, scales = (self.k, self.ks) if name == "k" else (self.v, self.vs)
        out = np.zeros((n, self.d))
        for i in range(0, n, P):
            pg = self.table[b, i // P]
            m = min(P, n - i)
            out[i:i + m] = E4M3[codes[pg, h, :m]] * 2.0 ** (int(scales[pg, h]) - 127)
        return out

    def _bounds(self, pg, h, n):
        c = E4M3[self.k[pg, h, :n]]
        self.kb[pg, h, 0] = e4m3_codes(c.min(0))
        self.kb[pg, h, 1] = e4m3_codes(c.max(0))

    def append(self, k, v, lens, n_new):
        """k, v: [B, H, T, d] float64, finite."""
        P = self.page
        for b in range(k.shape[0]):
            n = int(n_new[b])
            for pos in range(int(lens[b]) // P * P, int(lens[b]) + n, P):
                pg = self.table[b, pos // P]
                s0 = max(int(lens[b]) - pos, 0)
                s1 = min(P, int(lens[b]) + n - pos)
                if s1 <= s0:
                    continue
                i0 = pos + s0 - int(lens[b])
                for h in range(self.H):
                    for x, codes, scales in ((k, self.k, self.ks), (v, self.v, self.vs)):
                        new = x[b, h, i0:i0 + s1 - s0]
                        X = least_exponent(np.abs(new).max())
                        if s0:
                            X_old = int(scales[pg, h]) - 127
                            X = max(X, X_old)
                            codes[pg, h, :s0] = e4m3_codes(E4M3[codes[pg, h, :s0]] * 2.0 ** (X_old - X))
                        codes[pg, h, s0:s1] = e4m3_codes(new * 2.0 ** -X)
                        scales[pg, h] = X + 127
                    self._bounds(pg, h, s1)

    def sees(self, length, q_len, t, causal):
        return max(0, min(length, length - q_len + t + 1)) if causal else length

    def fwd(self, q, lens, q_lens, causal=True, scale=None, pages=None):
        """q [B, Hq, T, d] float64.  Returns (o, lse, spread, eps, small): spread
        = sum p |v| / sum p, eps = a bound of the error of a score per unit
        2^-23 * d (the greatest sum |q| |k| * scale), small = 2^-35 * keys * the
        largest |v| of the sequence's head."""
        B, Hq, T, d = q.shape
        G = Hq // self.H
        scale = d ** -0.5 if scale is None else scale
        o, spread = np.zeros(q.shape), np.zeros(q.shape)
        lse, eps, small = np.full((B, Hq, T), -np.inf), np.zeros((B, Hq, T)), np.zeros((B, Hq, T))
        for b in range(B):
            L, n = int(lens[b]), int(q_lens[b])
            for hk in range(self.H):
                K, V = self.read("k", b, hk, L), self.read("v", b, hk, L)
                for t in range(n):
                    see = np.arange(L) < self.sees(L, n, t, causal)
                    if pages is not None:
                        mine = pages[b, hk, t]
                        see &= np.isin(np.arange(L) // self.page, mine[mine >= 0])
                    if not see.any():
                        continue
                    for h in range(hk * G, hk * G + G):
                        s = K[see] @ q[b, h, t] * scale
                        m = s.max()
                        p = np.exp(s - m)
                        o[b, h, t] = p @ V[see] / p.sum()
                        spread[b, h, t] = p @ np.abs(V[see]) / p.sum()
                        lse[b, h, t] = m + np.log(p.sum())
                        eps[b, h, t] = (np.abs(K[see]) @ np.abs(q[b, h, t])).max() * scale
                        small[b, h, t] = 2.0 ** -35 * see.sum() * np.abs(V).max()
        return o, lse, spread, eps, small

    def select(self, q, lens, q_lens, n_sel):
        B, Hq, T, d = q.shape
        G, P = Hq // self.H, self.page
        out = np.full((B, self.H, T, n_sel), -1, dtype=np.int64)
        for b in range(B):
            L, n = int(lens[b]), int(q_lens[b])
            for hk in range(self.H):
                for t in range(n):
                    count = -(-self.sees(L, n, t, True) // P)
                    if not count:
                        continue
                    pg = self.table[b, :count]
                    kb = E4M3[self.kb[pg, hk]] * 2.0 ** (self.ks[pg, hk].astype(np.float64) - 127)[:, None, None]
                    x = q[b, hk * G:hk * G + G, t]
                    bound = (np.maximum(x, 0).sum(0) * kb[:, 1] + np.minimum(x, 0).sum(0) * kb[:, 0]).sum(1)
                    bound[count - 1] = np.inf
                    top = np.sort(np.argsort(-bound, kind="stable")[:n_sel])
                    out[b, hk, t, :len(top)] = top
        return out

    def weigh(self, q, lse, lens, q_lens, weight, causal=True, scale=None):
        B, Hq, T, d = q.shape
        G = Hq // self.H
        scale = d ** -0.5 if scale is None else scale
        out = np.array(weight, dtype=np.float64)
        for b in range(B):
            L, n = int(lens[b]), int(q_lens[b])
            for hk in range(self.H):
                K = self.read("k", b, hk, L)
                for t in range(n):
                    see = np.arange(L) < self.sees(L, n, t, causal)
                    for h in range(hk * G, hk * G + G):
                        if np.isfinite(lse[b, h, t]):
                            out[b, hk, :L][see] += np.exp(K[see] @ q[b, h, t] * scale - lse[b, h, t])
        return out

    def evict(self, lens, weight, dst, budget, recent):
        """Changes the pool; returns (new_lens, kept, weights)."""
        B, P = len(lens), self.page
        kept = np.full((B, self.H, budget), -1, dtype=np.int64)
        w_out = np.zeros((B, self.H, dst.shape[1] * P))
        src = Ref(self.k, self.v, self.ks, self.vs, self.kb, self.table)
        for b in range(B):
            L = int(lens[b])
            m = min(L, budget)
            for h in range(self.H):
                w = np.array(weight[b, h, :L], dtype=np.float64)
                w[np.isnan(w)] = -np.inf
                r = min(recent, m)         # kept whatever the others weigh, infinities included
                at = np.sort(np.concatenate([np.argsort(-w[:L - r], kind="stable")[:m - r], np.arange(L - r, L)]))
                kept[b, h, :m] = at
                w_out[b, h, :m] = weight[b, h, at]
                for name, codes, scales in (("k", self.k, self.ks), ("v", self.v, self.vs)):
                    x = src.read(name, b, h, L)[at]
                    for i in range(0, m, P):
                        pg = dst[b, i // P]
                        part = x[i:i + P]
                        X = least_exponent(np.abs(part).max())
                        codes[pg, h, :len(part)] = e4m3_codes(part * 2.0 ** -X)
                        scales[pg, h] = X + 127
                        if name == "k":
                            self._bounds(pg, h, len(part))
        return np.minimum(lens, budget), kept, w_out


def contents(cache):
    """The five tensors on the host, codes as values (so -0 equals 0)."""
    c = [t.cpu().numpy() for t in (cache.k, cache.v, cache.kb)]
    return [E4M3[x] for x in c] + [cache.ks.cpu().numpy(), cache.vs.cpu().numpy()]


def make(fa, lens, H, d, page, seed=0, device="cuda", room=0, k_scale=1.0, v_scale=1.0, stale=0xff, spare=3, first=0):
    """A cache with random tokens, its pages in random order behind `first`
    unused ones; every byte no token uses is `stale` (0xff: NaN)."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    per = max(1, max(-(-(int(n) + room) // page) for n in lens))
    n = B * per + spare + first
    cache = fa.cache_alloc(n, H, d, page, device)
    for t in (cache.k, cache.v, cache.kb, cache.ks, cache.vs):
        t[first:].fill_(stale if t.dim() == 4 else 200)
    table = (torch.randperm(B * per + spare, generator=g)[:B * per] + first).int().view(B, per).to(device)
    T = max(1, max(int(x) for x in lens))
    k = (torch.randn(B, H, T, d, generator=g) * k_scale).to(torch.bfloat16).to(device)
    v = (torch.randn(B, H, T, d, generator=g) * v_scale).to(torch.bfloat16).to(device)
    ln = torch.tensor([int(x) for x in lens], dtype=torch.int32, device=device)
    fa.cache_append(cache, k, v, table, torch.zeros_like(ln), n_new=ln)
    return cache, table, ln
