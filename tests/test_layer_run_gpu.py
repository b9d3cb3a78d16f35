"""The operators of a layer together, as they are used."""
import pytest
import torch

import layer_ref as ref
from gpu_util import rel_l2, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return require_gpu()


def grid(t, h, w):
    return torch.stack(torch.meshgrid(*(torch.arange(n) for n in (t, h, w)), indexing="ij")).flatten(1).int().cuda()


def test_video_block_inference(fa):
    """Fused projection -> norm and rotation on three axes -> FP4 self-attention -> norm -> attention to a text, eager
    and captured."""
    B, H, d, Nk = 2, 3, 128, 77
    pos = grid(3, 10, 7)
    N = pos.shape[1]
    g = torch.Generator(device="cuda").manual_seed(0)
    qkv = torch.randn((B, N, 3, H, d), generator=g, device="cuda").to(torch.bfloat16)
    text = torch.randn((B, Nk, 2, H, d), generator=g, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([77, 12], device="cuda", dtype=torch.int32)
    w = [1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in range(4)]
    sections = [22, 21, 21]
    freqs = fa.rope_freqs(d, sections)

    def block():
        q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
        q, k = fa.qk_norm_rope(q, k, pos, freqs, w[0], w[1], sections=sections, interleaved=True)
        o, _ = fa.fwd(*fa.quantize_qkv(q, k, v.contiguous()))
        x, _ = fa.qk_norm_rope(o, None, q_weight=w[2])
        tk, tv = (text[:, :, i].transpose(1, 2) for i in range(2))
        tk, _ = fa.qk_norm_rope(tk, None, q_weight=w[3])
        return q, k, x, tk, tv, *fa.cross_fwd(x, tk, tv, lens)

    q, k, x, tk, tv, o, lse = block()
    fa.sync_status()
    th = ref.turns(pos[None].expand(B, -1, -1), freqs, sections)
    ref.assert_within(q, *ref.norm_rope(qkv[:, :, 0].transpose(1, 2), w[0], th, True, True, 1e-6), "q")
    ref.assert_within(k, *ref.norm_rope(qkv[:, :, 1].transpose(1, 2), w[1], th, True, True, 1e-6), "k")
    want, bound, _, _ = ref.cross(x, tk, tv, lens)
    ref.assert_within(o, want, bound, "o")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = block()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, (q, k, x, tk, tv, o, lse)))


def test_training_step_of_cross_attention(fa):
    """Norm of q and k, attention, and the gradients back to what went in, against autograd in 64 bits."""
    B, Hq, Hkv, Nq, Nk, d = 2, 4, 2, 150, 90, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    xq = torch.randn((B, Nq, Hq, d), generator=g, device="cuda").to(torch.bfloat16).transpose(1, 2)
    kv = torch.randn((B, Nk, 2, Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    xk, v = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    wq, wk = (1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    lens = torch.tensor([90, 41], device="cuda", dtype=torch.int32)
    dout = torch.randn((B, Hq, Nq, d), generator=g, device="cuda").to(torch.bfloat16)

    q, _ = fa.qk_norm_rope(xq, None, q_weight=wq)
    k, _ = fa.qk_norm_rope(xk, None, q_weight=wk)
    o, lse = fa.cross_fwd(q, k, v, lens)
    dq, dk, dv = fa.cross_bwd(q, k, v, o, dout, lse, lens)
    dxq, _, dwq, _ = fa.qk_norm_rope_bwd(dq, None, xq, None, q_weight=wq)
    dxk, _, dwk, _ = fa.qk_norm_rope_bwd(dk, None, xk, None, q_weight=wk)
    fa.sync_status()

    leaf = lambda t: t.double().detach().requires_grad_()
    a, b, c, wa, wb = leaf(xq), leaf(xk), leaf(v), leaf(wq), leaf(wk)
    want = ref.cross(ref.norm_rope(a, wa, None, False, True, 1e-6)[0], ref.norm_rope(b, wb, None, False, True, 1e-6)[0],
                     c, lens)[0]
    want.backward(dout.double())
    # q, k, o, P, dS and each gradient are rounded to bf16 on the way, off by up to 2^-8 each, about 2^-8 / sqrt(3) of
    # the norm on average: eight of them in a row stay below 2^-8 * 8 / sqrt(3) = 0.018
    for name, x, y in (("o", o, want.detach()), ("dxq", dxq, a.grad), ("dxk", dxk, b.grad), ("dv", dv, c.grad),
                       ("dwq", dwq, wa.grad), ("dwk", dwk, wb.grad)):
        assert rel_l2(x.double().cpu(), y.cpu()) <= 0.018, name


def test_decoding_step(fa):
    """One token a sequence: rotation at its position, into the 8-bit cache, attention over it and to an encoder."""
    B, Hq, Hkv, d, T = 3, 8, 2, 128, 5
    g = torch.Generator(device="cuda").manual_seed(4)
    cache = fa.cache_alloc(B, Hkv, d, page=16)
    table = torch.arange(B, device="cuda", dtype=torch.int32)[:, None]
    lens = torch.zeros(B, device="cuda", dtype=torch.int32)
    enc = torch.randn((B, 33, 2, Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    freqs = fa.rope_freqs(d)
    start = torch.tensor([0, 100000, 7], device="cuda", dtype=torch.int32)
    ks, vs = [], []
    for t in range(T):
        qkv = torch.randn((B, 1, Hq + 2 * Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
        q, k, v = (x.transpose(1, 2) for x in qkv.split([Hq, Hkv, Hkv], 2))
        q, k = fa.qk_norm_rope(q, k, (start + t)[:, None, None].contiguous(), freqs)
        fa.cache_append(cache, k, v.contiguous(), table, lens)
        lens += 1
        o, _ = fa.cache_fwd(q, cache, table, lens)
        c, _ = fa.cross_fwd(q, enc[:, :, 0].transpose(1, 2), enc[:, :, 1].transpose(1, 2))
        ks.append(k)
        vs.append(v)
    fa.sync_status()
    # e4m3 is off by up to 2^-4 of a value, about 2^-4 / sqrt(12) of a norm, in K and in V
    want, _, _, _ = ref.cross(q, torch.cat(ks, 2), torch.cat(vs, 2))
    assert rel_l2(o.double().cpu(), want.cpu()) <= 2.0 ** -4
    want, bound, _, _ = ref.cross(q, enc[:, :, 0].transpose(1, 2), enc[:, :, 1].transpose(1, 2))
    ref.assert_within(c, want, bound, "cross")
