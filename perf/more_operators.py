"""Norm and rotation of queries and keys, and cross attention, as timed cases.

Every case is one pass through one operator: ``rope`` (per-head RMS norm of q
and k and the rotation by their positions on one or several axes), ``rope_bwd``
(its gradients, those of the norm's weights among them), ``cross`` (attention of
queries to the states of an encoder of another length) and ``cross_bwd`` (its
gradients).

``own = False`` runs each operator in elementary torch operations, ``own =
True`` through this package; both take the same state.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    c = []
    # one decoding step of a serving batch, far into long contexts: latency
    c.append(dict(name="rope_token", op="rope", B=64, Hq=32, Hkv=8, N=1, d=128, axes=1, pairs=False, far=500000))
    # the projections of a training step, two sequences of 8192 tokens
    c.append(dict(name="rope_train", op="rope", B=2, Hq=32, Hkv=8, N=8192, d=128, axes=1, pairs=False, far=0))
    # a video of 21 x 30 x 52 patches, positions on three axes
    c.append(dict(name="rope_video", op="rope", B=1, Hq=24, Hkv=24, N=32760, d=128, axes=3, pairs=True, far=0))
    # a few short prompts of an image and text model, heads of 64
    c.append(dict(name="rope_bwd_short", op="rope_bwd", B=3, Hq=14, Hkv=2, N=77, d=64, axes=3, pairs=False, far=0,
                  f32=False))
    # the training step's gradients, FP32 as the quantized backward gives them
    c.append(dict(name="rope_bwd_train", op="rope_bwd", B=2, Hq=32, Hkv=8, N=8192, d=128, axes=1, pairs=False, far=0,
                  f32=True))
    # a batch of decoding steps over encoder states of mixed lengths: bandwidth
    c.append(dict(name="cross_token", op="cross", B=64, Hq=16, Hkv=16, Nq=1, Nk=1500, d=64, ragged=True))
    # one user, a few drafted tokens over long states with shared heads: latency
    c.append(dict(name="cross_draft", op="cross", B=1, Hq=32, Hkv=8, Nq=3, Nk=16383, d=128, ragged=False))
    # image tokens attend to short captions: bandwidth again
    c.append(dict(name="cross_caption", op="cross", B=4, Hq=16, Hkv=16, Nq=4096, Nk=77, d=128, ragged=True))
    # the video's patches attend to a text of up to 512 tokens
    c.append(dict(name="cross_video", op="cross", B=1, Hq=24, Hkv=24, Nq=32760, Nk=512, d=128, ragged=False))
    # a text decoder's tokens and encoder states in training, heads of 64
    c.append(dict(name="cross_bwd_text", op="cross_bwd", B=8, Hq=16, Hkv=16, Nq=333, Nk=1500, d=64, ragged=True))
    # queries of many tokens share the heads of long states
    c.append(dict(name="cross_bwd_long", op="cross_bwd", B=2, Hq=32, Hkv=8, Nq=1024, Nk=4100, d=128, ragged=False))
    # the video and its text in training
    c.append(dict(name="cross_bwd_video", op="cross_bwd", B=1, Hq=24, Hkv=24, Nq=32760, Nk=512, d=128, ragged=False))
    return c


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "cross", "cross", "cross_bwd", "cross_bwd"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16, 24])
    G = rng.choice([1, 1, 2, 3, 4, 7, 8])
    Hq = max(1, min(Hkv * G, 32) // Hkv) * Hkv
    if op in ("rope", "rope_bwd"):
        N = 1 if rng.random() < 0.25 else _log(rng, 2, 32760)
        N = min(N, 786432 // (Hq + Hkv))
        most = max(1, min(64, 786432 // (N * (Hq + Hkv))))
        axes = rng.choice([1, 1, 2, 3])
        c = dict(op=op, B=_log(rng, 1, most), Hq=Hq, Hkv=Hkv, N=N, d=d, axes=axes, pairs=rng.random() < 0.5,
                 far=0 if axes > 1 or rng.random() < 0.5 else _log(rng, 1, 1000000))
        if op == "rope_bwd":
            c["f32"] = rng.random() < 0.5
        return c
    # scores of all heads: at most those of the video and its text
    room = 24 * 32760 * 512
    if op == "cross":
        Nq = rng.choice([1, 1, 2, 3, 5]) if rng.random() < 0.4 else _log(rng, 6, 32760)
        Nk = _log(rng, 1, min(16384, max(16, room // (Hq * Nq))))
        B = _log(rng, 1, max(1, min(64, room // (Hq * Nq * Nk), 100663296 // (Hkv * Nk * d))))
        while B * Hq * Nq * d > 24 * 32760 * 128 and B > 1:
            B -= 1
        Nq = min(Nq, 24 * 32760 * 128 // (B * Hq * d))
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, ragged=rng.random() < 0.5)
    Nq = _log(rng, 1, 24 * 32760 // Hq)
    Nk = _log(rng, 40, min(8192, max(80, room // (Hq * Nq))))
    Nq = min(Nq, room // (Hq * Nk))
    B = _log(rng, 1, max(1, min(32, room // (Hq * Nq * Nk), 24 * 32760 * 128 // (Hq * Nq * d),
                                50331648 // (Hkv * Nk * d))))
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, ragged=rng.random() < 0.5)


# ----------------------------------------------------------------------------
# state
# ----------------------------------------------------------------------------
def _sections(case):
    """Channel pairs that turn with each axis: of several axes the first takes the rest of an even division."""
    h, a = case["d"] // 2, case["axes"]
    return [h - (a - 1) * (h // a)] + [h // a] * (a - 1)


def _freqs(case):
    """Radians a position, [d / 2] in 64 bits on the host: each axis has a ladder of its own."""
    return torch.cat([10000.0 ** (-torch.arange(n, dtype=torch.float64) / n) for n in _sections(case)])


def _positions(case, g):
    """int32 [B, axes, N]: tokens in a row from somewhere up to `far` (one axis), or the patches of a grid."""
    B, N, a = case["B"], case["N"], case["axes"]
    i = torch.arange(N, device=DEV)
    if a == 1:
        start = torch.randint(0, case["far"] + 1, (B, 1, 1), generator=g, device=DEV)
        return (start + i).int()
    side = 52 if a == 3 else 128
    parts = [i // (side * 30), i // side % 30, i % side] if a == 3 else [i // side, i % side]
    return torch.stack(parts).int().expand(B, -1, -1).contiguous()


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    st = dict(case=case)
    if case["op"] in ("rope", "rope_bwd"):
        N = case["N"]
        # views of one fused projection [B, N, (Hq + 2 Hkv) d], a few channels much larger than the others
        x = torch.randn((B, N, Hq + 2 * Hkv, d), generator=g, device=DEV) * 2.0
        x[..., : d // 32] *= 6.0
        x = x.to(torch.bfloat16)
        st["q"], st["k"] = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq: Hq + Hkv].transpose(1, 2)
        st["wq"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
        st["wk"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
        st["pos"], st["freqs"], st["sections"] = _positions(case, g), _freqs(case), _sections(case)
        if case["op"] == "rope_bwd":
            dt = torch.float32 if case["f32"] else torch.bfloat16
            st["dyq"] = torch.randn((B, Hq, N, d), generator=g, device=DEV).to(dt)
            st["dyk"] = torch.randn((B, Hkv, N, d), generator=g, device=DEV).to(dt)
        return st
    Nq, Nk = case["Nq"], case["Nk"]
    st["q"] = _randn(g, B, Hq, Nq, d)
    # views of one projection of the encoder's states [B, Nk, 2, Hkv, d]
    kv = _randn(g, B, Nk, 2, Hkv, d)
    st["k"], st["v"] = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    st["lens"] = None
    if case["ragged"]:
        st["lens"] = torch.randint(max(1, Nk // 8), Nk + 1, (B,), generator=g, device=DEV).int()
    if case["op"] == "cross_bwd":
        o, st["lse"] = _cross(st)
        st["o"] = o.to(torch.bfloat16)
        st["do"] = _randn(g, B, Hq, Nq, d)
    return st


# ----------------------------------------------------------------------------
# the operators in elementary operations
# ----------------------------------------------------------------------------
def _cos_sin(st):
    """[B, 1, N, d / 2] each; the angles in 64 bits."""
    freqs = st["freqs"].to(DEV)
    axis = torch.repeat_interleave(torch.arange(len(st["sections"])), torch.tensor(st["sections"])).to(DEV)
    angle = st["pos"].double()[:, axis].transpose(1, 2) * freqs
    return torch.cos(angle)[:, None].float(), torch.sin(angle)[:, None].float()


def _split(x, pairs):
    return (x[..., 0::2], x[..., 1::2]) if pairs else x.chunk(2, -1)


def _join(a, b, pairs):
    return torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)


def _rope_one(x, w, cs, pairs):
    x = x.float()
    a, b = _split(x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w, pairs)
    return _join(a * cs[0] - b * cs[1], b * cs[0] + a * cs[1], pairs).to(torch.bfloat16)


def _rope_bwd_one(dy, x, w, cs, pairs):
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xr = x * r
    a, b = _split(dy.float(), pairs)
    g = _join(a * cs[0] + b * cs[1], b * cs[0] - a * cs[1], pairs)
    u = g * w
    dx = r * (u - xr * (u * xr).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (g * xr).sum((0, 1, 2), dtype=torch.float64).float()


def _scores(st):
    """FP32 scores [B, Hkv, G Nq, Nk], -inf behind a sequence's keys."""
    q, k = st["q"], st["k"]
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    s = torch.matmul(q.float().reshape(B, Hkv, Hq // Hkv * Nq, d), k.float().transpose(2, 3)) / math.sqrt(d)
    if st["lens"] is not None:
        s = s.masked_fill(torch.arange(Nk, device=DEV) >= st["lens"][:, None, None, None], -math.inf)
    return s


def _cross(st):
    """FP32 o [B, Hq, Nq, d] and lse [B, Hq, Nq]."""
    B, Hq, Nq, d = st["q"].shape
    s = _scores(st)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m)
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e, st["v"].float()) / l
    return o.reshape(B, Hq, Nq, d), (m + torch.log(l)).reshape(B, Hq, Nq)


def _cross_bwd(st):
    B, Hq, Nq, d = st["q"].shape
    Hkv = st["k"].shape[1]
    rows = lambda x: x.float().reshape(B, Hkv, Hq // Hkv * Nq, -1)  # noqa: E731
    p = torch.exp(_scores(st) - rows(st["lse"]))
    dp = torch.matmul(rows(st["do"]), st["v"].float().transpose(2, 3))
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(d)
    dv = torch.matmul(p.transpose(2, 3), rows(st["do"]))
    dk = torch.matmul(ds.transpose(2, 3), rows(st["q"]))
    dq = torch.matmul(ds, st["k"].float()).reshape(B, Hq, Nq, d)
    return dq.to(torch.bfloat16), dk.to(torch.bfloat16), dv.to(torch.bfloat16)


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def _own(st):
    import precision_attention_fa4fp4_gb300 as fa
    case = st["case"]
    if case["op"] == "rope":
        return fa.qk_norm_rope(st["q"], st["k"], st["pos"], st["freqs"], st["wq"], st["wk"], sections=st["sections"],
                               interleaved=case["pairs"], eps=EPS)
    if case["op"] == "rope_bwd":
        return fa.qk_norm_rope_bwd(st["dyq"], st["dyk"], st["q"], st["k"], st["pos"], st["freqs"], st["wq"], st["wk"],
                                   sections=st["sections"], interleaved=case["pairs"], eps=EPS)
    if case["op"] == "cross":
        return fa.cross_fwd(st["q"], st["k"], st["v"], kv_lens=st["lens"])
    return fa.cross_bwd(st["q"], st["k"], st["v"], st["o"], st["do"], st["lse"], kv_lens=st["lens"])


def run(st):
    if own:
        return _own(st)
    case = st["case"]
    if case["op"] == "rope":
        cs = _cos_sin(st)
        return _rope_one(st["q"], st["wq"], cs, case["pairs"]), _rope_one(st["k"], st["wk"], cs, case["pairs"])
    if case["op"] == "rope_bwd":
        cs = _cos_sin(st)
        dq, dwq = _rope_bwd_one(st["dyq"], st["q"], st["wq"], cs, case["pairs"])
        dk, dwk = _rope_bwd_one(st["dyk"], st["k"], st["wk"], cs, case["pairs"])
        return dq, dk, dwq, dwk
    if case["op"] == "cross":
        o, lse = _cross(st)
        return o.to(torch.bfloat16), lse
    return _cross_bwd(st)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    if case["op"] in ("rope", "rope_bwd"):
        n = B * (Hq + Hkv) * case["N"] * d
        if case["op"] == "rope":
            return dict(bytes=4 * n + 4 * B * case["axes"] * case["N"], flops=8 * n)
        return dict(bytes=(8 if case["f32"] else 6) * n + 4 * B * case["axes"] * case["N"], flops=18 * n)
    Nq, Nk = case["Nq"], case["Nk"]
    L = (max(1, Nk // 8) + Nk) / 2 if case["ragged"] else Nk          # keys of an average sequence
    rows, keys = B * Hq * Nq, B * Hkv * L
    if case["op"] == "cross":
        return dict(bytes=rows * (4 * d + 4) + 4 * keys * d, flops=4 * rows * L * d)
    return dict(bytes=rows * (8 * d + 4) + 4 * keys * d + 4 * B * Hkv * Nk * d, flops=10 * rows * L * d)


# ----------------------------------------------------------------------------
# the operators in 64 bits, from their definitions, a head at a time
# ----------------------------------------------------------------------------
def _turn64(x, st, b, pairs, back):
    """One head's rows [N, d] turned by their positions (back: the other way)."""
    d = x.shape[-1]
    out = x.clone()
    i = 0
    for axis, n in enumerate(st["sections"]):
        for _ in range(n):
            th = st["pos"][b, axis].double() * float(st["freqs"][i])
            if back:
                th = -th
            p, q = (2 * i, 2 * i + 1) if pairs else (i, i + d // 2)
            out[:, p] = x[:, p] * torch.cos(th) - x[:, q] * torch.sin(th)
            out[:, q] = x[:, p] * torch.sin(th) + x[:, q] * torch.cos(th)
            i += 1
    return out


def exact(case, seed):
    st = prepare(case, seed)
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    if case["op"] in ("rope", "rope_bwd"):
        outs, weights = [], []
        for name in ("q", "k"):
            w = st["w" + name].double()
            H, N = st[name].shape[1], case["N"]
            out = torch.empty((B, H, N, d), dtype=torch.float64, device=DEV)
            dw = torch.zeros(d, dtype=torch.float64, device=DEV)
            for b in range(B):
                # all of a sequence's heads at once: rows [H N, d] under the positions repeated
                x = st[name][b].double().reshape(H * N, d)
                one = dict(sections=st["sections"], freqs=st["freqs"], pos=st["pos"][b: b + 1].repeat(1, 1, H))
                size = torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
                if case["op"] == "rope":
                    y = _turn64(x / size * w, one, 0, case["pairs"], False)
                else:
                    g = _turn64(st["dy" + name][b].double().reshape(H * N, d), one, 0, case["pairs"], True)
                    dw += (g * x / size).sum(0)
                    u = g * w
                    y = u / size - x * (u * x).sum(-1, keepdim=True) / (d * size ** 3)
                out[b] = y.reshape(H, N, d)
            outs.append(out)
            weights.append(dw)
        return tuple(outs) if case["op"] == "rope" else tuple(outs + weights)
    Nq, Nk, G = case["Nq"], case["Nk"], Hq // Hkv
    new = lambda *s: torch.zeros(s, dtype=torch.float64, device=DEV)  # noqa: E731
    o, lse = new(B, Hq, Nq, d), new(B, Hq, Nq)
    dq, dk, dv = new(B, Hq, Nq, d), new(B, Hkv, Nk, d), new(B, Hkv, Nk, d)
    for b in range(B):
        L = Nk if st["lens"] is None else int(st["lens"][b])
        for h in range(Hq):
            K, V = st["k"][b, h // G, :L].double(), st["v"][b, h // G, :L].double()
            Q = st["q"][b, h].double()
            s = Q @ K.T * d ** -0.5
            z = torch.logsumexp(s, -1)
            P = torch.exp(s - z[:, None])
            if case["op"] == "cross":
                o[b, h], lse[b, h] = P @ V, z
                continue
            dO = st["do"][b, h].double()
            dP = dO @ V.T
            dS = P * (dP - (dO * (P @ V)).sum(-1, keepdim=True)) * d ** -0.5
            dq[b, h] = dS @ K
            dk[b, h // G, :L] += dS.T @ Q
            dv[b, h // G, :L] += P.T @ dO
    return (o, lse) if case["op"] == "cross" else (dq, dk, dv)


if __name__ == "__main__":
    r = random.Random(0)
    for c in listed() + [draw(r) for _ in range(6)]:
        print(c, work(c))
