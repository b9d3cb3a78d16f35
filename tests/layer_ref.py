"""Plain forms in 64 bits of the norm and rotation of queries and keys and of cross
attention, with elementwise error bounds.

A rounding to bf16 is off by at most half a step, 2^-8 of the value (U).  Bounds
count those of the results and of P and dS, to which the kernels round for their
products; what FP32 adds (sums, the native sine, cosine and exponential, 2^-21 or
better each) is bounded by a small multiple of the magnitudes that are summed."""
import torch

U = 2.0 ** -8


def turns(positions, freqs, sections):
    """Angles [B, 1, N, d/2] of positions [B, axes, N]."""
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).to(positions.device)
    return (positions.double()[:, axis].transpose(1, 2) * freqs.to(positions.device))[:, None]


def split(x, interleaved):
    return (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)


def join(a, b, interleaved):
    return torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)


def turn(x, th, interleaved):
    if th is None:
        return x
    a, b = split(x, interleaved)
    return join(a * th.cos() - b * th.sin(), b * th.cos() + a * th.sin(), interleaved)


def norm_rope(x, w, th, interleaved, norm, eps):
    """(y, bound on a kernel's error)."""
    x = x.double()
    n = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() if norm else x
    n = n * w.double() if w is not None else n
    y = turn(n, th, interleaved)
    a, b = split(n.abs(), interleaved)
    return y, U * y.abs() + 2.0 ** -19 * join(a + b, a + b, interleaved) + 1e-38


def norm_rope_bwd(dy, x, w, th, interleaved, norm, eps):
    """(dx, its bound, dw, its bound)."""
    x = x.double()
    g = turn(dy.double(), None if th is None else -th, interleaved)
    a, b = split(dy.double().abs(), interleaved)
    size = join(a + b, a + b, interleaved)
    if not norm:
        return g, U * g.abs() + 2.0 ** -19 * size, None, None
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    w = torch.ones(x.shape[-1], device=x.device) if w is None else w
    u, xr = g * w.double(), x * r
    dx = r * (u - xr * (u * xr).mean(-1, keepdim=True))
    us = size * w.double().abs()
    slack = r * (us + xr.abs() * (us * xr.abs()).mean(-1, keepdim=True))
    return (dx, U * dx.abs() + 2.0 ** -17 * slack + 1e-38, (g * xr).sum((0, 1, 2)),
            2.0 ** -18 * (size * xr.abs()).sum((0, 1, 2)) + 1e-30)


def _parts(q, k, lens, scale):
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    scale = d ** -0.5 if scale <= 0 else scale
    there = torch.ones(B, Nk, dtype=torch.bool, device=q.device)
    if lens is not None:
        there = torch.arange(Nk, device=q.device) < lens[:, None].clamp(0, Nk)
    # what lies behind a sequence's keys does not count, NaN or not
    K = k.double().masked_fill(~there[:, None, :, None], 0)
    return B, Hq, Nq, d, Hkv, Nk, scale, there[:, None, None, :], K


def cross(q, k, v, lens=None, scale=0.0):
    """(o, bound, lse, bound)."""
    B, Hq, Nq, d, Hkv, Nk, scale, there, K = _parts(q, k, lens, scale)
    V = v.double().masked_fill(~there[:, 0, 0, :, None][:, None], 0)
    Q = q.double().reshape(B, Hkv, Hq // Hkv * Nq, d)
    s = (Q @ K.transpose(2, 3) * scale).masked_fill(~there, -float("inf"))
    lse = torch.logsumexp(s, -1) if Nk else torch.full(s.shape[:3], -float("inf"), dtype=torch.float64, device=q.device)
    p = torch.exp(s - lse[..., None]).nan_to_num(0.0) * there
    # a score's error: d products summed in FP32, the tensor cores' sums cut (2^-23)
    es = (Q.abs() @ K.abs().transpose(2, 3) * scale * (d * 2.0 ** -23)).masked_fill(~there, 0.0)
    worst = es.amax(-1, keepdim=True) if Nk else torch.zeros(*s.shape[:3], 1, dtype=torch.float64, device=q.device)
    size = p @ V.abs()
    o = p @ V
    bound = U * o.abs() + (U + 2.0 ** -12 + 2 * worst) * size + 1e-38
    shape = (B, Hq, Nq)
    return (o.reshape(*shape, d), bound.reshape(*shape, d), lse.reshape(shape),
            (worst[..., 0] + 2.0 ** -20 * (1 + lse.abs().nan_to_num(posinf=0.0))).reshape(shape))


def cross_bwd(q, k, v, o, dout, lse, lens=None, scale=0.0):
    """((dq, bound), (dk, bound), (dv, bound)) for the o and lse given."""
    B, Hq, Nq, d, Hkv, Nk, scale, there, K = _parts(q, k, lens, scale)
    V = v.double().masked_fill(~there[:, 0, 0, :, None][:, None], 0)
    rows = lambda x: x.double().reshape(B, Hkv, Hq // Hkv * Nq, -1)
    Q, G, O, L = rows(q), rows(dout), rows(o), rows(lse)
    use = there & (L > -float("inf"))
    p = torch.exp((Q @ K.transpose(2, 3) * scale - L).masked_fill(~use, -float("inf")))
    ep = p * ((Q.abs() @ K.abs().transpose(2, 3) * scale) * (d * 2.0 ** -23) + 2.0 ** -19 * (1 + L.abs().nan_to_num(posinf=0.0)))
    dp, D = G @ V.transpose(2, 3), (G * O).sum(-1, keepdim=True)
    # below 2^-126 the native exponential gives 0, and so may the rounding of dS: P is off by 2^-126 more, dS by that
    # and by what the P makes of it (d S = P (dP - D))
    least = use * 2.0 ** -126
    ep = ep + least
    edp = ((G.abs() @ V.abs().transpose(2, 3)) + (G * O).abs().sum(-1, keepdim=True)) * (d * 2.0 ** -23)
    ds = p * (dp - D)
    eds = U * ds.abs() + (1 + U) * (ep * (dp - D).abs() + p * edp) + least
    few = 1 + 2.0 ** -10        # sums in FP32
    out = []
    for x, e, y in ((ds, eds, K), (ds.transpose(2, 3), eds.transpose(2, 3), Q)):
        t = scale * (x @ y)
        out.append((t, U * t.abs() + few * scale * (e @ y.abs()) + 2.0 ** -14 * scale * (x.abs() @ y.abs()) + 1e-38))
    t = p.transpose(2, 3) @ G
    out.append((t, U * t.abs() + few * ((U * p + ep).transpose(2, 3) @ G.abs()) + 2.0 ** -14 * (p.transpose(2, 3) @ G.abs())
                + 1e-38))
    dq, dk, dv = out
    return tuple(x.reshape(B, Hq, Nq, d) for x in dq), dk, dv


def assert_within(got, want, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    off = (got - want).abs()
    over = off / bound
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times its bound at {tuple(int(i) for i in (over == over.max()).nonzero()[0])}"
